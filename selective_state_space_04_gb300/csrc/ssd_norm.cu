// ssd_norm.cu -- RMSNorm over a token's whole row: with the residual's addition
// in front or a SiLU gate behind, out in the input's type or as 8-bit whole
// numbers with a scale; and its gradients.
//
// A row is read once and stays in registers: thread i of the row's group holds
// the vectors (8 elements) i, i + group, ...  Forward, with h = x + residual:
//   v = h r w (SiLU(z)),  r = 1 / sqrt(mean h^2 + eps)
// The 8-bit form needs max|v| over the row; v is r times t = h w (SiLU(z)) and r
// is one number, so sum h^2 and max|t| are reduced together, and
//   q = rint(t * 127 / max|t|),   scale = r max|t| / 127.
// The maximum is taken over the bit patterns of |t|, in which an infinity or NaN
// is above every finite number and is not lost as it is by fmaxf.
//
// Bound by memory: 32768 rows of 2560 with a residual, bf16, take 95 us (104% of a plain copy's rate), their
// gradients 111 (89%); 16384 such rows in fp32 96 us (103%) and 107 (92%).  Into 8 bits, 8192 rows of 2560 with an fp32
// residual take 37.5 us (91%).  The gated form reaches 60% (4096 rows of 5120: 25.6 us; with z at an odd offset, read
// element by element, 30.8).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpRowDim = 1024;   // rows up to here are one warp's, 4 vectors a lane at most
constexpr int kWarpRows = 8;        // rows (warps) of such a block
constexpr float kTiny = 1.17549435e-38f;   // 2^-126

enum Mode { kPlain, kResidual, kGate };

struct NormParams {
    const void *x, *res, *z;
    const float *w;
    void *out, *ro;
    int8_t *q;
    float *qs;
    long long rows;
    long long xs, rs, zs, os, ros, qst;   // row strides, elements
    int D;
    float eps;
    bool zvec;                       // z's rows are 16-byte aligned
};

// 8 consecutive elements as they lie in memory
template <typename T> struct Vec {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const void *p, long long at)
    {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + at);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            u[i] = __ldcs(s + i);
    }
    // the same from any alignment of T's
    __device__ __forceinline__ void load_any(const void *p, long long at)
    {
        const T *s = static_cast<const T *>(p) + at;
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = s[i];
        memcpy(u, v, sizeof(u));
    }
    __device__ __forceinline__ void store(void *p, long long at) const
    {
        uint4 *d = reinterpret_cast<uint4 *>(static_cast<T *>(p) + at);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            __stcs(d + i, u[i]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t v[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(v[i] << 16);
                f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                f[4 * i] = __uint_as_float(u[i].x);
                f[4 * i + 1] = __uint_as_float(u[i].y);
                f[4 * i + 2] = __uint_as_float(u[i].z);
                f[4 * i + 3] = __uint_as_float(u[i].w);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                v[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
            u[0] = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                u[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                                  __float_as_uint(f[4 * i + 3]));
        }
    }
};

// (not through the read-only path: the launch before may write the weights while this one lives)
__device__ __forceinline__ void load_w(const float *w, int v, float (&f)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(w)[2 * v], b = reinterpret_cast<const float4 *>(w)[2 * v + 1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(ss / D + eps); 0 for a row of zeros with eps 0, so that it stays zero
__device__ __forceinline__ float inv_rms(float ss, int D, float eps)
{
    const float m = ss / (float)D + eps;
    return m == 0.f ? 0.f : 1.f / sqrtf(m);
}

// v sigmoid(v) from the approximate exponential and reciprocal (a few units of 2^-23 and |v| of 2^-24;
// five instructions: this and the rounding below took the gated norm of 4096 rows of 5120 from 28.2 us to 25.6).  Below
// about -87.3, where the reciprocal is under 2^-126, the result is 0 (at most 2^-119 off).
__device__ __forceinline__ float silu(float v)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return v * r;
}

// VPT: vectors a thread holds.  kWarp: a row is one warp's, else one block's.
template <typename T, typename R, int kMode, bool kQ8, int VPT, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kMaxThreads) ssd_norm_kernel(NormParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float part[kMaxThreads / 32];
    __shared__ uint32_t top[kMaxThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = kWarp ? lane : threadIdx.x, group = kWarp ? 32 : blockDim.x;
    const long long row = kWarp ? (long long)blockIdx.x * kWarpRows + warp : blockIdx.x;
    if (kWarp && row >= p.rows)
        return;
    const int nv = p.D / 8;
    float h[VPT][8], w[VPT][8];
    {
        Vec<T> ux[VPT], uz[VPT];
        Vec<R> ur[VPT];
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
            if (v < nv) {
                ux[a].load(p.x, row * p.xs + 8 * v);
                if (kMode == kResidual)
                    ur[a].load(p.res, row * p.rs + 8 * v);
                if (kMode == kGate) {
                    if (p.zvec)
                        uz[a].load(p.z, row * p.zs + 8 * v);
                    else
                        uz[a].load_any(p.z, row * p.zs + 8 * v);
                }
            }
        }
#pragma unroll
        for (int a = 0; a < VPT; ++a)
            if (tid + a * group < nv)
                load_w(p.w, tid + a * group, w[a]);
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[a][e] = 0.f;
            if (v >= nv)
                continue;
            ux[a].get(h[a]);
            if (kMode == kResidual) {
                float f[8];
                ur[a].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[a][e] += f[e];
                if (p.ro) {
                    Vec<R> u;
                    u.set(h[a]);
                    u.store(p.ro, row * p.ros + 8 * v);
                }
            }
            if (kMode == kGate) {
                float f[8];
                uz[a].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[a][e] *= silu(f[e]);
            }
        }
    }
    float ss = 0.f;
    uint32_t most = 0u;
#pragma unroll
    for (int a = 0; a < VPT; ++a) {
        if (tid + a * group >= nv)
            continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(h[a][e], h[a][e], ss);
            if (kQ8) {
                h[a][e] *= w[a][e];
                most = max(most, __float_as_uint(h[a][e]) & 0x7fffffffu);
            }
        }
    }
    ss = warp_sum(ss);
    if (kQ8)
        most = __reduce_max_sync(0xffffffffu, most);
    if (!kWarp) {
        if (lane == 0) {
            part[warp] = ss;
            top[warp] = most;
        }
        __syncthreads();
        const int nw = blockDim.x >> 5;
        ss = warp_sum(lane < nw ? part[lane] : 0.f);
        if (kQ8)
            most = __reduce_max_sync(0xffffffffu, lane < nw ? top[lane] : 0u);
    }
    const float r = inv_rms(ss, p.D, p.eps);
    if (kQ8) {
        const float m = __uint_as_float(most);
        float scale = r * m / 127.f, by = 127.f / m;
        if (!(scale <= 3.4028235e38f) || !(m <= 3.4028235e38f)) {   // an infinity or NaN in the row, or a product past fp32
            scale = __uint_as_float(0x7fffffffu);
            by = 0.f;
        } else if (scale < kTiny || m < kTiny) {   // (products below 2^-126 have lost bits)
            scale = by = 0.f;
        } else if (m < 127.f * kTiny) {   // the quotient would leave the range: both by 2^32
            by = 127.f / (m * 4294967296.f);
#pragma unroll
            for (int a = 0; a < VPT; ++a)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[a][e] *= 4294967296.f;
        }
        if (tid == 0)
            p.qs[row] = scale;
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
            if (v >= nv)
                continue;
            // 1.5 x 2^23 + x has the nearest whole number to x (even ones at halves) in its lowest bits;
            // conversions would share the exponentials' pipe
            uint32_t b[2] = {0u, 0u};
            if (by != 0.f)
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    uint32_t u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        u[i] = __float_as_uint(fmaf(h[a][e + i], by, 12582912.f));
                    b[e / 4] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
                }
            *reinterpret_cast<uint2 *>(p.q + row * p.qst + 8 * v) = make_uint2(b[0], b[1]);
        }
    } else {
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
            if (v >= nv)
                continue;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = h[a][e] * r * w[a][e];
            Vec<T> u;
            u.set(o);
            u.store(p.out, row * p.os + 8 * v);
        }
    }
}

template <typename K, typename... A>
cudaError_t launch_after(K *kernel, unsigned grid, unsigned threads, cudaStream_t st, const A &...args)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

template <typename T, typename R, int kMode, bool kQ8>
cudaError_t norm_launch_t(const NormParams &p, cudaStream_t st)
{
    const int nv = p.D / 8;
    if (p.D <= kWarpRowDim) {
        const unsigned grid = (unsigned)((p.rows + kWarpRows - 1) / kWarpRows);
        if (nv <= 32)
            return launch_after(ssd_norm_kernel<T, R, kMode, kQ8, 1, true>, grid, 32 * kWarpRows, st, p);
        if (nv <= 64)
            return launch_after(ssd_norm_kernel<T, R, kMode, kQ8, 2, true>, grid, 32 * kWarpRows, st, p);
        return launch_after(ssd_norm_kernel<T, R, kMode, kQ8, 4, true>, grid, 32 * kWarpRows, st, p);
    }
    const int vpt = nv <= 512 ? 1 : 2;   // (one vector up to 1024 threads was not measured)
    const unsigned threads = (unsigned)(((nv + vpt - 1) / vpt + 31) / 32 * 32);
    if (vpt == 1)
        return launch_after(ssd_norm_kernel<T, R, kMode, kQ8, 1, false>, (unsigned)p.rows, threads, st, p);
    return launch_after(ssd_norm_kernel<T, R, kMode, kQ8, 2, false>, (unsigned)p.rows, threads, st, p);
}

template <typename T, typename R>
cudaError_t norm_launch_types(const NormArgs &a, const NormParams &p, cudaStream_t st)
{
    const bool q8 = a.q != nullptr;
    if (a.z)
        return norm_launch_t<T, T, kGate, true>(p, st);
    if (a.residual)
        return q8 ? norm_launch_t<T, R, kResidual, true>(p, st) : norm_launch_t<T, R, kResidual, false>(p, st);
    return q8 ? norm_launch_t<T, T, kPlain, true>(p, st) : norm_launch_t<T, T, kPlain, false>(p, st);
}

// ---- gradients --------------------------------------------------------------

struct NormBwdParams {
    const void *h, *dout, *dres;
    const float *w;
    void *dx;
    float *part;   // [blocks][D], or null
    long long rows;
    long long hs, ds, rs, xs;
    int D;
    float eps;
};

constexpr int kBwdWarpRows = 8, kBwdThreads = 512;
constexpr int kBwdWarpDim = 512;   // rows up to here are one warp's, 2 vectors a lane at most

// Blocks (warps where a row is one warp's) take rows blockIdx, blockIdx + grid, ..., the next row's
// loads under way while one is summed and written; the weight's gradient is summed in registers over a
// block's rows and written as one partial row per block, which a second launch adds in block order.
template <typename T, typename R, bool kRes, int VPT, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kBwdWarpRows : kBwdThreads, kWarp || VPT > 1 || sizeof(R) > 2 ? 1 : 2) ssd_norm_bwd_kernel(NormBwdParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr bool kAhead = VPT < 4;   // (more would not fit the registers)
    __shared__ float2 part[2][kBwdThreads / 32];
    __shared__ __align__(16) float sums[kWarp ? kBwdWarpRows * kBwdWarpDim : 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = kWarp ? lane : threadIdx.x, group = kWarp ? 32 : blockDim.x;
    const int nv = p.D / 8;
    const float dim = (float)p.D;
    float w[VPT][8], acc[VPT][8];
#pragma unroll
    for (int a = 0; a < VPT; ++a) {
        if (tid + a * group < nv)
            load_w(p.w, tid + a * group, w[a]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[a][e] = 0.f;
    }
    const long long first = kWarp ? (long long)blockIdx.x * kBwdWarpRows + warp : blockIdx.x;
    const long long step = kWarp ? (long long)gridDim.x * kBwdWarpRows : gridDim.x;
    Vec<R> uh[VPT], ur[VPT], nh[VPT], nr[VPT];
    Vec<T> ud[VPT], nd[VPT];
    auto load = [&](long long row, Vec<R> (&h)[VPT], Vec<T> (&d)[VPT], Vec<R> (&r)[VPT]) {
        if (row >= p.rows)
            return;
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
            if (v < nv) {
                h[a].load(p.h, row * p.hs + 8 * v);
                d[a].load(p.dout, row * p.ds + 8 * v);
                if (kRes)
                    r[a].load(p.dres, row * p.rs + 8 * v);
            }
        }
    };
    if (kAhead)
        load(first, nh, nd, nr);
    int turn = 0;
    for (long long row = first; row < p.rows; row += step) {
        if (kAhead) {
#pragma unroll
            for (int a = 0; a < VPT; ++a) {
                uh[a] = nh[a];
                ud[a] = nd[a];
                if (kRes)
                    ur[a] = nr[a];
            }
            load(row + step, nh, nd, nr);
        } else {
            load(row, uh, ud, ur);
        }
        float ss = 0.f, c = 0.f;
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            if (tid + a * group >= nv)
                continue;
            float h[8], d[8];
            uh[a].get(h);
            ud[a].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(h[e], h[e], ss);
                c = fmaf(d[e] * w[a][e], h[e], c);
            }
        }
        ss = warp_sum(ss);
        c = warp_sum(c);
        if (!kWarp) {   // two turns' sums in turn: one barrier a row
            if (lane == 0)
                part[turn][warp] = make_float2(ss, c);
            __syncthreads();
            const float2 t = lane < (int)(blockDim.x >> 5) ? part[turn][lane] : make_float2(0.f, 0.f);
            ss = warp_sum(t.x);
            c = warp_sum(t.y);
            turn ^= 1;
        }
        const float r = inv_rms(ss, p.D, p.eps);
        const float k = r * c / dim;   // (h r is of the order of 1; r r would be infinite where rows are tiny and eps is 0)
#pragma unroll
        for (int a = 0; a < VPT; ++a) {
            const int v = tid + a * group;
            if (v >= nv)
                continue;
            float h[8], d[8], f[8], o[8];
            uh[a].get(h);
            ud[a].get(d);
            if (kRes)
                ur[a].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = h[e] * r, dx = r * (d[e] * w[a][e] - n * k);
                o[e] = kRes ? dx + f[e] : dx;
                acc[a][e] = fmaf(d[e], n, acc[a][e]);
            }
            Vec<R> u;
            u.set(o);
            u.store(p.dx, row * p.xs + 8 * v);
        }
    }
    if (!p.part)
        return;
    float *to = p.part + (size_t)blockIdx.x * p.D;
#pragma unroll
    for (int a = 0; a < VPT; ++a) {
        const int v = tid + a * group;
        if (v >= nv)
            continue;
        float4 *at = reinterpret_cast<float4 *>(kWarp ? sums + warp * kBwdWarpDim : to) + 2 * v;
        at[0] = make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
        at[1] = make_float4(acc[a][4], acc[a][5], acc[a][6], acc[a][7]);
    }
    if (kWarp) {   // the block's warps in order
        __syncthreads();
        for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kBwdWarpRows; ++j)
                s += sums[j * kBwdWarpDim + i];
            to[i] = s;
        }
    }
}

// dweight = the sum of n partial rows: block = 32 columns, warp y the rows y, y + 32, ...
__global__ void __launch_bounds__(1024) ssd_norm_dweight_kernel(const float *part, float *dw, int n, int D)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float s[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float t = 0.f;
    if (col < D) {
#pragma unroll 4
        for (int i = y; i < n; i += 32)
            t += part[(size_t)i * D + col];
    }
    s[y][threadIdx.x & 31] = t;
    __syncthreads();
    t = warp_sum(s[threadIdx.x & 31][y]);
    const int out = blockIdx.x * 32 + y;
    if ((threadIdx.x & 31) == 0 && out < D)
        dw[out] = t;
}

// vectors a thread holds, and threads of a row; of fp32 rows two, where one would be 512 threads: their
// registers are what fits on an SM.  Four vectors (rows above 8192) have no room for the next row's loads, and with
// fp32 rows some registers go to local memory: 4096 rows of 16384 take 110 us in bf16 and 256 in fp32 (72 and 62% of a
// plain copy's rate), 8192 rows of 8192 89 and 168 (88 and 94%).
int bwd_threads(const ssd_norm_dims_t &d, int *vpt)
{
    const int nv = d.dim / 8;
    *vpt = nv <= (d.residual_dtype == SSD_DTYPE_F32 ? kBwdThreads / 2 : kBwdThreads) ? 1 : nv <= 2 * kBwdThreads ? 2 : 4;
    return ((nv + *vpt - 1) / *vpt + 31) / 32 * 32;
}

// Blocks: as many as run at once (1024 threads an SM, measured best on the one width that was tried: on 32768 rows of 2560 three blocks
// of 320 take 111 us, two 125, four 134; where a row is a warp's, two blocks of 256 of them), but
// eight rows each (per warp) where that fills the SMs: a block's partial sums cost as much as a row.
int bwd_blocks(const ssd_norm_dims_t &d)
{
    if (d.rows <= 0)
        return 0;
    int vpt;
    const bool warp = d.dim <= kBwdWarpDim;
    const int per_sm = warp ? 2 : std::max(1, 1024 / bwd_threads(d, &vpt));
    const int64_t rows = warp ? (d.rows + kBwdWarpRows - 1) / kBwdWarpRows : d.rows;
    return (int)std::min<int64_t>({rows, std::max<int64_t>(sm_count(), (rows + 7) / 8), (int64_t)sm_count() * per_sm});
}

template <typename T, typename R, bool kRes>
cudaError_t bwd_launch_t(const NormBwdParams &p, const ssd_norm_dims_t &d, int blocks, cudaStream_t st)
{
    if (p.D <= kBwdWarpDim) {
        if (p.D <= 256)
            return launch_after(ssd_norm_bwd_kernel<T, R, kRes, 1, true>, blocks, 32 * kBwdWarpRows, st, p);
        return launch_after(ssd_norm_bwd_kernel<T, R, kRes, 2, true>, blocks, 32 * kBwdWarpRows, st, p);
    }
    int vpt;
    const unsigned threads = bwd_threads(d, &vpt);
    if (vpt == 1)
        return launch_after(ssd_norm_bwd_kernel<T, R, kRes, 1, false>, blocks, threads, st, p);
    if (vpt == 2)
        return launch_after(ssd_norm_bwd_kernel<T, R, kRes, 2, false>, blocks, threads, st, p);
    return launch_after(ssd_norm_bwd_kernel<T, R, kRes, 4, false>, blocks, threads, st, p);
}

template <typename T, typename R>
cudaError_t bwd_launch_types(const NormBwdParams &p, const ssd_norm_dims_t &d, int blocks, cudaStream_t st)
{
    return p.dres ? bwd_launch_t<T, R, true>(p, d, blocks, st) : bwd_launch_t<T, R, false>(p, d, blocks, st);
}

}  // namespace

cudaError_t norm_launch(const NormArgs &a, cudaStream_t st)
{
    SSD_NVTX_RANGE("norm_launch");
    if (a.d.rows == 0)
        return cudaSuccess;
    NormParams p;
    p.x = a.x;
    p.res = a.residual;
    p.z = a.z;
    p.w = a.weight;
    p.out = a.out;
    p.ro = a.residual_out;
    p.q = a.q;
    p.qs = a.q_scale;
    p.rows = a.d.rows;
    p.xs = a.d.x_stride;
    p.rs = a.d.residual_stride;
    p.zs = a.d.z_stride;
    p.os = a.d.out_stride;
    p.ros = a.d.ro_stride;
    p.qst = a.d.q_stride;
    p.D = a.d.dim;
    p.eps = a.d.eps;
    p.zvec = ((uintptr_t)a.z & 15) == 0 && (p.rows == 1 || p.zs * (a.d.dtype == SSD_DTYPE_F32 ? 4 : 2) % 16 == 0);
    if (a.d.dtype == SSD_DTYPE_F32)
        return norm_launch_types<float, float>(a, p, st);
    return a.d.residual_dtype == SSD_DTYPE_F32 ? norm_launch_types<__nv_bfloat16, float>(a, p, st)
                                               : norm_launch_types<__nv_bfloat16, __nv_bfloat16>(a, p, st);
}

size_t norm_bwd_workspace_bytes(const ssd_norm_dims_t &d) { return (size_t)bwd_blocks(d) * d.dim * 4; }

cudaError_t norm_bwd_launch(const NormBwdArgs &a, void *workspace, cudaStream_t st)
{
    SSD_NVTX_RANGE("norm_bwd_launch");
    if (a.d.rows == 0)
        return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.d.dim * 4, st) : cudaSuccess;
    NormBwdParams p;
    p.h = a.h;
    p.dout = a.dout;
    p.dres = a.dres;
    p.w = a.weight;
    p.dx = a.dx;
    p.part = a.dweight ? static_cast<float *>(workspace) : nullptr;
    p.rows = a.d.rows;
    p.hs = a.d.ro_stride;
    p.ds = a.d.x_stride;
    p.rs = a.d.residual_stride;
    p.xs = a.d.out_stride;
    p.D = a.d.dim;
    p.eps = a.d.eps;
    const int blocks = bwd_blocks(a.d);
    cudaError_t e;
    if (a.d.dtype == SSD_DTYPE_F32)
        e = bwd_launch_types<float, float>(p, a.d, blocks, st);
    else
        e = a.d.residual_dtype == SSD_DTYPE_F32 ? bwd_launch_types<__nv_bfloat16, float>(p, a.d, blocks, st)
                                                : bwd_launch_types<__nv_bfloat16, __nv_bfloat16>(p, a.d, blocks, st);
    if (e != cudaSuccess || !a.dweight)
        return e;
    return launch_after(ssd_norm_dweight_kernel, (unsigned)((p.D + 31) / 32), 1024, st, (const float *)p.part, a.dweight, blocks, p.D);
}

}  // namespace ssd
