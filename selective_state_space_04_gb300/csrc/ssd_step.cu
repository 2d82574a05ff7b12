// ssd_step.cu -- the causal conv1d + SiLU and the scan for one token of each of
// several sequences, their states in a pool of slots.
//
// Per row and head: u = SiLU(bias + sum of K taps) for the head's P channels and its
// group's 2 N, then one step of the recurrence as in ssd_decode.cu:
//   h[p,n] = dA h[p,n] + dt B[n] x[p],   y[p] = sum_n C[n] h[p,n] + D x[p]
// What bounds it is the fp32 state, P N 4 bytes in and out per row and head; the
// convolution's inputs are a few hundredths of that.  So a block of 4 warps takes one
// head of one row, or several of a group where their states are small, issues the loads of its first
// state rows, and convolves while they are on their way: every block computes its group's B and C
// itself, which costs K loads from the caches per channel and saves a launch.  (The next rows' loads into
// the registers of the row just stored: 111 us for 125 sequences of 80 heads of 64 x 128, 105 without.  Today they take
// 100 us, 96% of a plain copy's rate; one sequence takes 4.8.)
//
// The sequences' last inputs are a ring of K entries, entry p mod K for position p:
// the token's own input goes into the entry that held position t - K, which no tap
// reads, so that the blocks of one row need no order among them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kLoads = 8;   // 16-byte loads of a lane (for NV = 1) in flight together, as in ssd_decode.cu

struct StepParams {
    const void *xbc, *dt_raw;
    void *ring, *y;
    const float *w, *bias, *dt_bias, *A_log, *D;
    float *states;
    const int32_t *slots, *positions;
    long long nslots, xs, ds, ys;
    int H, P, N, G, K, C, hc;   // hc: heads of a block, a divisor of H / G
    uint32_t mul, sh;           // row / P = (row * mul) >> sh for the rows of a block
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// SiLU(conv) of channel c.  `in`: the token's inputs, `ring`: the slot's K entries.
template <typename T, int K>
__device__ __forceinline__ float convolved(const T *in, const T *ring, const float *w, const float *bias, int c, int C, int t)
{
    float u = bias ? bias[c] : 0.f;
    u = fmaf(w[(size_t)c * K], to_f32<T>(in[c]), u);
#pragma unroll
    for (int j = 1; j < K; ++j)
        if (t >= j)
            u = fmaf(w[(size_t)c * K + j], to_f32<T>(ring[(size_t)((t - j) % K) * C + c]), u);
    return u / (1.f + expf(-u));
}

// A state row is 4 LPR NV elements at most: LPR lanes with NV pieces of 4 each, 32 / LPR rows side by side in
// a warp (NV > 1 with whole warps only).
template <typename T, typename TD, int LPR, int NV, int K, bool kHeads>
__global__ void __launch_bounds__(kWarps * 32, NV == 1 ? 6 : 1) ssd_step_kernel(StepParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ float conv[];   // x [hc P], B [N], C [N]; dt, dA and D per head, of several
    constexpr int kSide = 32 / LPR, kPass = kLoads * kSide;   // rows of a warp at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, col = 4 * (lane % LPR);
    const int H = p.H, P = p.P, N = p.N, C = p.C, hc = kHeads ? p.hc : 1, R = hc * P, blocks = kHeads ? H / hc : H;
    float *heads = conv + R + 2 * N;
    const long long i = blockIdx.x / blocks;
    const int h0 = (int)(blockIdx.x - i * blocks) * hc, per = H / p.G, g = h0 / per;
    const long long slot = p.slots[i];
    const int t = p.positions[i];
    T *y = static_cast<T *>(p.y) + i * p.ys + (long long)h0 * P;
    if (slot < 0 || slot >= p.nslots || t < 0) {
        for (int c = threadIdx.x; c < R; c += kWarps * 32)
            y[c] = from_f32<T>(0.f);
        return;
    }
    float *state = p.states + ((size_t)slot * H + h0) * P * N + (size_t)sub * N + col;
    float4 hv[kLoads][NV];
    auto load = [&](int p0) {
#pragma unroll
        for (int r = 0; r < kLoads; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                hv[r][k] = t > 0 && p0 + r * kSide + sub < R && col + 128 * k < N
                               ? __ldcs(reinterpret_cast<const float4 *>(state + (size_t)(p0 + r * kSide) * N + 128 * k))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(warp * kPass);

    const T *in = static_cast<const T *>(p.xbc) + i * p.xs;
    T *ring = static_cast<T *>(p.ring) + (size_t)slot * K * C;
    T *mine = ring + (size_t)(t % K) * C;
    const int x0 = h0 * P, b0 = H * P + g * N, c0 = H * P + p.G * N + g * N;
    for (int c = threadIdx.x; c < R + 2 * N; c += kWarps * 32) {
        const int ch = c < R ? x0 + c : c < R + N ? b0 + c - R : c0 + c - R - N;
        conv[c] = convolved<T, K>(in, ring, p.w, p.bias, ch, C, t);
        if (c < R || h0 == g * per)   // the group's first head keeps B and C
            mine[ch] = in[ch];
    }
    float dt = 0.f, dA = 0.f, Dh = 0.f;
    for (int j = kHeads ? threadIdx.x : 0; j < hc; j += kWarps * 32) {
        const int h = h0 + j;
        const float z = to_f32<TD>(static_cast<const TD *>(p.dt_raw)[i * p.ds + h]) + p.dt_bias[h];
        dt = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
        dA = expf(dt * -expf(p.A_log[h]));
        Dh = p.D[h];
        if (kHeads) {
            heads[3 * j] = dt;
            heads[3 * j + 1] = dA;
            heads[3 * j + 2] = Dh;
        }
    }
    __syncthreads();

    float bv[NV][4], cv[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = col + 128 * k + e;
            bv[k][e] = n < N ? conv[R + n] : 0.f;
            cv[k][e] = n < N ? conv[R + N + n] : 0.f;
        }
    for (int p0 = warp * kPass; p0 < R; p0 += kWarps * kPass) {
        if (p0 != warp * kPass)
            load(p0);
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
            const int pr = p0 + r * kSide + sub;
            if (kHeads && pr < R) {
                const float *head = heads + 3 * (int)(((uint64_t)(uint32_t)pr * p.mul) >> p.sh);
                dt = head[0];
                dA = head[1];
                Dh = head[2];
            }
            const float x = pr < R ? conv[pr] : 0.f, dtx = dt * x;
            float acc = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float4 &v = hv[r][k];
                v.x = fmaf(dA, v.x, dtx * bv[k][0]);
                v.y = fmaf(dA, v.y, dtx * bv[k][1]);
                v.z = fmaf(dA, v.z, dtx * bv[k][2]);
                v.w = fmaf(dA, v.w, dtx * bv[k][3]);
                acc = fmaf(cv[k][0], v.x, acc);
                acc = fmaf(cv[k][1], v.y, acc);
                acc = fmaf(cv[k][2], v.z, acc);
                acc = fmaf(cv[k][3], v.w, acc);
                if (pr < R && col + 128 * k < N)
                    __stcs(reinterpret_cast<float4 *>(state + (size_t)(p0 + r * kSide) * N + 128 * k), v);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (col == 0 && pr < R)
                y[pr] = from_f32<T>(fmaf(Dh, x, acc));
        }
    }
}

template <typename T, typename TD, int LPR, int NV, int K, bool kHeads>
cudaError_t launch_heads(const StepParams &p, unsigned grid, cudaStream_t st)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = (size_t)(p.hc * p.P + 2 * p.N + 3 * p.hc) * 4;
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ssd_step_kernel<T, TD, LPR, NV, K, kHeads>, p);
}

// (several heads: where a head's states are half a block's share, so N <= 128 only)
template <typename T, typename TD, int LPR, int NV, int K>
cudaError_t launch_k(const StepParams &p, unsigned grid, cudaStream_t st)
{
    if constexpr (NV == 1)
        if (p.hc > 1)
            return launch_heads<T, TD, LPR, NV, K, true>(p, grid, st);
    return launch_heads<T, TD, LPR, NV, K, false>(p, grid, st);
}

template <typename T, typename TD, int LPR, int NV>
cudaError_t launch_row(const StepParams &p, unsigned grid, cudaStream_t st)
{
    return p.K == 2   ? launch_k<T, TD, LPR, NV, 2>(p, grid, st)
           : p.K == 3 ? launch_k<T, TD, LPR, NV, 3>(p, grid, st)
                      : launch_k<T, TD, LPR, NV, 4>(p, grid, st);
}

template <typename T, typename TD>
cudaError_t launch_t(const StepParams &p, unsigned grid, cudaStream_t st)
{
    if (p.N <= 32)
        return p.N <= 16 ? launch_row<T, TD, 4, 1>(p, grid, st) : launch_row<T, TD, 8, 1>(p, grid, st);
    if (p.N <= 128)
        return p.N <= 64 ? launch_row<T, TD, 16, 1>(p, grid, st) : launch_row<T, TD, 32, 1>(p, grid, st);
    return p.N <= 256 ? launch_row<T, TD, 32, 2>(p, grid, st) : launch_row<T, TD, 32, 4>(p, grid, st);
}

}  // namespace

cudaError_t step_launch(const StepArgs &a, cudaStream_t st)
{
    SSD_NVTX_RANGE("step_launch");
    if (a.d.rows == 0)
        return cudaSuccess;
    StepParams p;
    p.xbc = a.xbc;
    p.dt_raw = a.dt_raw;
    p.ring = a.ring;
    p.y = a.y;
    p.w = a.weight;
    p.bias = a.bias;
    p.dt_bias = a.dt_bias;
    p.A_log = a.A_log;
    p.D = a.D;
    p.states = a.states;
    p.slots = a.slots;
    p.positions = a.positions;
    p.nslots = a.d.nslots;
    p.xs = a.d.xbc_stride;
    p.ds = a.d.dt_stride;
    p.ys = a.d.y_stride;
    p.H = a.d.nheads;
    p.P = a.d.headdim;
    p.N = a.d.dstate;
    p.G = a.d.ngroups;
    p.K = a.d.kernel_size;
    p.C = p.H * p.P + 2 * p.G * p.N;
    // Heads of a block: up to 32 KB of states, as long as every SM has eight blocks.  (512 sequences of 80 heads
    // of 64 x 16: a head each 133 us, 8 KB 101, 16 KB 81, 32 KB 78, 64 KB 82.)
    p.hc = 1;
    const int per = p.H / p.G;
    for (int n = 2; n <= per && p.N <= 128 && (long long)n * p.P * p.N <= 8192 && a.d.rows * (p.H / n) >= 8 * sm_count(); ++n)
        if (per % n == 0)
            p.hc = n;
    p.sh = 31;   // exact for rows below 2^31 (P <= 2^31)
    while ((1u << (p.sh - 31)) < (uint32_t)p.P)
        ++p.sh;
    p.mul = (uint32_t)((1ull << p.sh) / (uint32_t)p.P + 1);
    const unsigned grid = (unsigned)(a.d.rows * (p.H / p.hc));
    cudaError_t e;
    if (a.d.dtype == SSD_DTYPE_F32)
        e = launch_t<float, float>(p, grid, st);
    else
        e = a.d.dt_dtype == SSD_DTYPE_F32 ? launch_t<__nv_bfloat16, float>(p, grid, st) : launch_t<__nv_bfloat16, __nv_bfloat16>(p, grid, st);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
