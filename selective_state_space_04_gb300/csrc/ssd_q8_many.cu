// ssd_q8_many.cu -- the 8-bit product for many tokens, bound by the tensor cores.
//
// Two launches.  The first widens both operands to fp16 (exactly: see ssd_q8_mid.cu) into
// scratch, as the images of the tiles that the second reads: 128 rows x 64 inner
// elements, 16 KB, swizzled, in the order of use, so that a tile is one contiguous copy
// (the tokens' slab by slab, all of them in a row, so that a tile may have any number of them).
// It moves 3 bytes per element of the operands, a few percent of the product's time where
// there are many tokens, and takes all work but copies out of the second.
//
// The second: pairs of CTAs (cta_group::2) on tiles of 256 channels x up to 256 tokens.  Each
// CTA holds its half of the channels' and of the tokens' operand, so that a slab of 64
// inner elements is at most 32 KB of copies per CTA for 512 clocks of MMA.  The tensor pipe is busy 83% of the
// time at 8192 tokens of 10576 x 2560 (both launches 254 to 260 us, 1.75 to 1.71 PFLOP/s; repeated without a pause the
// power limit holds the clock near 1.78 GHz and it is 282 us), 71% at 4096 of 2560 x 5120.  Accumulators take
// 1024 inner elements each, as in ssd_q8_mid.cu, two of them in turn: while one is
// filled, eight warps add the other to 32-bit integers in registers (128 per thread).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "ssd_internal.h"
#include "ssd_q8.h"

namespace ssd {

using namespace ptx;

static __device__ unsigned int g_q8_many_error;

namespace {

constexpr int kImage = kQ8Image;
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * kImage;
constexpr int kChunkSlabs = 16;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;   // warps 0-7: results, 8: copies, 9: MMA (leader) or its relay
constexpr int kSmem = kStages * kStageBytes + 1024;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr long long kPanel = 32768;   // tokens widened at once: bounds their scratch (the weights' is 2 N K bytes)

enum { BAR_FULL = 0, BAR_EMPTY = kStages, BAR_ACC = 2 * kStages, BAR_DRAINED = BAR_ACC + 2, kBars = BAR_DRAINED + 2 };

__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_test(bar, parity))
                return true;
    } while (globaltimer_ns() - t0 < kTimeoutNs);
    atomicCAS(&g_q8_many_error, 0u, (unsigned)SSD_ERR_TIMEOUT);
    return false;
}
// bounded wait; false after kTimeoutNs
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity)
{
    return mbar_test(bar, parity) || wait_long(bar, parity);
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, wait_bar(bar, parity));
}

// The ring's next place, and the parity of its present use.  (Single threads walk the ring, and their
// instructions count: a division by the ring's size at each slab was a tenth of its time.)
struct Place {
    uint32_t s = 0, parity = 0;
    // the next
    __device__ __forceinline__ void next()
    {
        if (++s == kStages) {
            s = 0;
            parity ^= 1;
        }
    }
};

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Widens the weights' slabs (the first `wslabs`: tile by tile, slab by slab; none on later
// panels and for the tokens alone) and the panel's tokens'.  One block per image, 8 lanes a row
// with 8 elements each, so that a warp's stores are whole 128-byte rows (16
// elements a lane, two stores with a gap between: 23 us for 4096 tokens and 10576 x 2560
// weights).
__global__ void __launch_bounds__(256) ssd_q8_widen_kernel(const Q8Params p, uint8_t *wi, uint8_t *ai, long long wslabs, long long slabs)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    for (long long i = blockIdx.x; i < slabs; i += gridDim.x) {
        uint2 u[4];
        uint8_t *image;
        if (i < wslabs) {
            image = wi + i * kImage;
#pragma unroll
            for (int h = 0; h < 4; ++h)
                u[h] = *reinterpret_cast<const uint2 *>(p.w + i * 8192 + (c >> 1) * 2048 + (r0 + 32 * h) * 16 + (c & 1) * 8);
        } else {
            const long long j = i - wslabs, t0 = j / p.k64 * 128, k = j % p.k64;
            const int k0 = (int)k * 64 + c * 8;
            image = ai + (k * p.padded() + t0) * 128;
#pragma unroll
            for (int h = 0; h < 4; ++h)
                u[h] = load8(p, t0 + r0 + 32 * h, k0);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t f[4];
            widen4(u[h].x, f);
            widen4(u[h].y, f + 2);
            *reinterpret_cast<uint4 *>(image + sw128(r0 + 32 * h, c)) = make_uint4(f[0], f[1], f[2], f[3]);
        }
    }
}

// Lane l of 8 holds (as pairs, lower half first) its column of an 8 x 8 matrix of 16-bit values; it gets row l.
__device__ __forceinline__ uint4 transpose8(const uint32_t (&v)[4], int lane)
{
    // rows 4 .. 7 against rows 0 .. 3 of the lane 4 on
    uint32_t a[4], b[4];
    const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
    uint32_t s0 = __shfl_xor_sync(0xffffffffu, h4 ? v[0] : v[2], 4), s1 = __shfl_xor_sync(0xffffffffu, h4 ? v[1] : v[3], 4);
    // a[0..1]: rows (0,1),(2,3) (+4 if h4) of the lower lane of the pair, a[2..3]: of the upper
    a[0] = h4 ? s0 : v[0], a[1] = h4 ? s1 : v[1], a[2] = h4 ? v[2] : s0, a[3] = h4 ? v[3] : s1;
    s0 = __shfl_xor_sync(0xffffffffu, h2 ? a[0] : a[1], 2), s1 = __shfl_xor_sync(0xffffffffu, h2 ? a[2] : a[3], 2);
    // b[c]: the row pair of this lane's row, of columns c0 = lane & 1, c0 + 2, c0 + 4, c0 + 6
    b[0] = h2 ? s0 : a[0], b[1] = h2 ? a[1] : s0, b[2] = h2 ? s1 : a[2], b[3] = h2 ? a[3] : s1;
    uint32_t r[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, b[c], 1);
        // columns 2 c and 2 c + 1: of an even lane, its own and the other's lower halves
        r[c] = h1 ? __byte_perm(o, b[c], 0x7632) : __byte_perm(b[c], o, 0x5410);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// tile index -> (channel pair, token pair): 8 token pairs wide, channel pairs within
__device__ __forceinline__ void tile_at(int i, int cp, int tp, int &c, int &t)
{
    const int band = i / (8 * cp), in = i - band * 8 * cp, wide = min(8, tp - 8 * band);
    c = in / wide;
    t = 8 * band + in - c * wide;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ssd_q8_many_kernel(const Q8Params p, const uint8_t *wi, const uint8_t *ai, int tn, int cp, int tp)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kBars];
    __shared__ uint32_t holder;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pairs = gridDim.x >> 1, me = blockIdx.x >> 1, items = cp * tp;
    const int chunks = (p.k64 + kChunkSlabs - 1) / kChunkSlabs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars[BAR_FULL + i], rank == 0 ? 2 : 1);   // own copies; in the leader the other CTA's too
            mbar_init(&bars[BAR_EMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[BAR_ACC + i], 1);
            mbar_init(&bars[BAR_DRAINED + i], 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    cluster_sync();
    if (warp == 9) {
        tmem_alloc2(&holder, 512);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = holder;
    cluster_sync();   // both CTAs' tensor memory and barriers are there
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 8) {
        const bool issue = elect_one();
        const size_t slab = (size_t)p.padded() * 128;
        uint32_t n = 0;   // slabs so far
        Place at;
        bool ok = true;
        for (int i = me; i < items && ok; i += pairs) {
            int c, t;
            tile_at(i, cp, tp, c, t);
            const uint8_t *w = wi + (size_t)min(2 * c + (int)rank, p.tiles - 1) * p.k64 * kImage;
            // (rows past the tokens', in the last tile, are another slab's or the scratch's end)
            const uint8_t *a = ai + ((size_t)t * tn + rank * (tn / 2)) * 128;
            for (int k = 0; k < p.k64; ++k, ++n, at.next(), w += kImage, a += slab) {
                if (n >= kStages && !(ok = warp_wait(&bars[BAR_EMPTY + at.s], at.parity ^ 1)))
                    break;
                if (issue) {
                    mbar_arrive_expect_tx(&bars[BAR_FULL + at.s], kImage + tn * 64);
                    bulk_load(smem + at.s * kStageBytes, w, kImage, &bars[BAR_FULL + at.s]);
                    bulk_load(smem + at.s * kStageBytes + kImage, a, tn * 64, &bars[BAR_FULL + at.s]);
                }
                __syncwarp();
            }
        }
        // no copy may be under way when shared memory is given up (each stage's last phase)
        for (uint32_t j = n > kStages ? n - kStages : 0; j < n; ++j)
            wait_bar(&bars[BAR_FULL + j % kStages], (j / kStages) & 1);
        __syncwarp();
    } else if (warp == 9) {
        if (rank == 0) {
            const bool issue = elect_one();
            const uint32_t idesc = idesc_f16_f32(256, tn);
            const uint64_t a0 = sdesc_sw128(smem_u32(smem), 16, 1024);   // (descriptors count 16 bytes)
            uint32_t m = 0;   // accumulators so far
            Place at;
            bool ok = true;
            for (int i = me; i < items && ok; i += pairs)
                for (int ch = 0; ch < chunks && ok; ++ch, ++m) {
                    const uint32_t b = m & 1, acc = tmem + 256 * b;
                    if (m >= 2 && !(ok = warp_wait(&bars[BAR_DRAINED + b], (m / 2 - 1) & 1)))
                        break;
                    tc_fence_after();
                    const int n = min(kChunkSlabs, p.k64 - ch * kChunkSlabs);
                    for (int k = 0; k < n; ++k, at.next()) {
                        if (!(ok = warp_wait(&bars[BAR_FULL + at.s], at.parity)))
                            break;
                        tc_fence_after();
                        const uint64_t d = a0 + at.s * (kStageBytes / 16);
                        if (issue) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma2_ss(acc, d + 2 * kk, d + kImage / 16 + 2 * kk, idesc, kk > 0 ? 1u : (uint32_t)(k > 0));
                            mma2_commit(&bars[BAR_EMPTY + at.s]);
                        }
                        __syncwarp();
                    }
                    if (issue)
                        mma2_commit(&bars[BAR_ACC + b]);
                    __syncwarp();
                }
            // no MMA may be in flight when the pair gives its memories up: each accumulator's last
            for (uint32_t j = m > 2 ? m - 2 : 0; j < m; ++j)
                wait_bar(&bars[BAR_ACC + (j & 1)], (j / 2) & 1);
        } else if (lane == 0) {
            // this CTA's copies, told to the leader
            Place at;
            bool ok = true;
            for (int i = me; i < items && ok; i += pairs)
                for (int k = 0; k < p.k64 && ok; ++k, at.next())
                    if ((ok = wait_bar(&bars[BAR_FULL + at.s], at.parity)))
                        mbar_arrive_at(&bars[BAR_FULL + at.s], 0);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = warp >> 2;
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + tn / 2 * half;
        uint32_t m = 0;
        bool ok = true;
        for (int i = me; i < items && ok; i += pairs) {
            int c, t;
            tile_at(i, cp, tp, c, t);
            const int channel = (2 * c + (int)rank) * 128 + 32 * q + lane;
            const long long t0 = (long long)tn * t + tn / 2 * half;
            int acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j)
                acc[j] = 0;
            for (int ch = 0; ch < chunks; ++ch, ++m) {
                const uint32_t b = m & 1;
                if (lane == 0)   // (32 lanes that ask keep shared memory busy)
                    ok = wait_bar(&bars[BAR_ACC + b], (m / 2) & 1);
                if (!(ok = __shfl_sync(0xffffffffu, ok, 0)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 128; j += 16) {
                    if (j >= tn / 2)
                        break;
                    uint32_t v[16];
                    tmem_ld16(from + 256 * b + j, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[j + e] += __float2int_rn(__uint_as_float(v[e]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_at(&bars[BAR_DRAINED + b], 0);
            }
            if (!ok)
                break;
            const bool mine = channel < p.N;
            const float ws = mine ? p.ws[channel] : 0.f;
            const int left = (int)max(0ll, min((long long)(tn / 2), p.M - t0));
            // whole 16-byte pieces of the result's rows, where they are that and all channels are there
            const int ch0 = channel - lane;
            if (sizeof(T) == 2 && p.yvec && ch0 + 32 <= p.N) {
                // 8 tokens of 8 lanes' channels are transposed among the lanes: lane l gets token l's
                T *y = static_cast<T *>(p.y) + (t0 + (lane & 7)) * p.sy + ch0 + (lane & 24);
#pragma unroll
                for (int j = 0; j < 128; j += 8) {
                    if (j >= left)
                        break;
                    const float as = j + (lane & 7) < left ? p.as[t0 + j + (lane & 7)] : 0.f;
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = (float)acc[j + e] * __shfl_sync(0xffffffffu, as, e, 8) * ws;
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
                    const uint4 u = transpose8(v, lane);
                    if (j + (lane & 7) < left)
                        __stcs(reinterpret_cast<uint4 *>(y + j * p.sy), u);
                }
            } else {
                T *y = static_cast<T *>(p.y) + t0 * p.sy + channel;
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (mine && j < left)
                        y[j * p.sy] = from_f32<T>((float)acc[j] * p.as[t0 + j] * ws);
            }
        }
    }
    tc_fence_before();
    cluster_sync();   // neither CTA reads the other's memories any more
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

cudaLaunchConfig_t after(cudaLaunchAttribute (&pdl)[1], cudaStream_t st)
{
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T>
cudaError_t many_t(const Q8Params &p, uint8_t *ws, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(ssd_q8_many_kernel<T>, kSmem, done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute pdl[1];
    cudaLaunchConfig_t cfg = after(pdl, st);
    const long long wslabs = (long long)p.tiles * p.k64;
    uint8_t *ai = ws + wslabs * kImage;
    for (long long m0 = 0; m0 < p.M; m0 += kPanel) {
        Q8Params q = p;
        q.M = std::min(kPanel, p.M - m0);
        q.a = p.a + m0 * p.sa;
        q.as = p.as + m0;
        q.y = static_cast<T *>(p.y) + m0 * p.sy;
        const int cp = (p.tiles + 1) / 2, pairs = sm_count() / 2;
        // Tokens of a tile: the pairs take tiles in waves, and a slab's time goes by its bytes, 16 KB of
        // weights and 64 a token.  (160 tiles of 256 tokens are 3 waves of 76, the third almost
        // empty; 220 of 192 are 3 shorter ones: 4096 tokens of 2560 x 5120 95 -> 80 us.)
        int tn = 256;
        long long best = INT64_MAX;
        for (int n = 256; n >= 64; n -= 32) {
            const long long cost = ((q.M + n - 1) / n * cp + pairs - 1) / pairs * (256 + n);
            if (cost < best) {
                best = cost;
                tn = n;
            }
        }
        const int tp = (int)((q.M + tn - 1) / tn);
        e = q8_widen_launch(q, ws, ai, m0 == 0 ? wslabs : 0, st);
        if (e != cudaSuccess)
            return e;
        cfg.gridDim = dim3(2 * (unsigned)std::min<long long>((long long)cp * tp, pairs));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        e = cudaLaunchKernelEx(&cfg, ssd_q8_many_kernel<T>, q, (const uint8_t *)ws, (const uint8_t *)ai, tn, cp, tp);
        if (e != cudaSuccess)
            return e;
        note_launches(1);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t q8_widen_launch(const Q8Params &p, uint8_t *wi, uint8_t *ai, long long wslabs, cudaStream_t st)
{
    const long long slabs = wslabs + (p.M + 127) / 128 * p.k64;
    cudaLaunchAttribute pdl[1];
    cudaLaunchConfig_t cfg = after(pdl, st);
    cfg.gridDim = dim3((unsigned)std::min<long long>(slabs, 1 << 16));
    cfg.blockDim = dim3(256);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ssd_q8_widen_kernel, p, wi, ai, wslabs, slabs);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

size_t q8_many_workspace_bytes(const Q8Params &p)
{
    // (the last tile's copies end up to 256 rows behind the tokens')
    return ((size_t)p.tiles + (size_t)((std::min(kPanel, p.M) + 127) / 128)) * p.k64 * kImage + 256 * 128;
}

cudaError_t q8_many_launch(const Q8Params &p, bool f32, void *workspace, cudaStream_t st)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return f32 ? many_t<float>(p, ws, st) : many_t<__nv_bfloat16>(p, ws, st);
}

ssd_status_t q8_many_read_device_error(uint32_t *code)
{
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_q8_many_error, sizeof(v)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_q8_many_error, &zero, sizeof(zero)) != cudaSuccess)
        return SSD_ERR_CUDA;
    *code = v;
    return SSD_OK;
}

}  // namespace ssd
