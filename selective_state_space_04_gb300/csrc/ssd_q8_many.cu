// ssd_q8_many.cu -- the 8-bit product for many tokens, bound by the tensor cores.
//
// Two launches.  The first widens both operands to fp16 (exactly: see ssd_q8_mid.cu) into
// scratch, as the images of the tiles that the second reads: 128 rows x 64 inner
// elements, 16 KB, swizzled, in the order of use, so that a tile is one contiguous copy.
// It moves 3 bytes per element of the operands, a few percent of the product's time where
// there are many tokens, and takes all work but copies out of the second.
//
// The second: pairs of CTAs (cta_group::2) on tiles of 256 channels x 256 tokens.  Each
// CTA holds its 128 rows of the channels' and of the tokens' operand, so that a slab of 64
// inner elements is 32 KB of copies per CTA for 512 clocks of MMA.  Accumulators take
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
constexpr long long kPanel = 32768;   // tokens widened at once: bounds the scratch

enum { BAR_FULL = 0, BAR_EMPTY = kStages, BAR_ACC = 2 * kStages, BAR_DRAINED = BAR_ACC + 2, kBars = BAR_DRAINED + 2 };

// bounded wait; false after kTimeoutNs
__device__ bool wait_bar(uint64_t *bar, uint32_t parity)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_test(bar, parity))
            return true;
    const uint64_t t0 = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_test(bar, parity))
                return true;
    } while (globaltimer_ns() - t0 < kTimeoutNs);
    atomicCAS(&g_q8_many_error, 0u, (unsigned)SSD_ERR_TIMEOUT);
    return false;
}

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
                u[h] = __ldg(reinterpret_cast<const uint2 *>(p.w + i * 8192 + (c >> 1) * 2048 + (r0 + 32 * h) * 16 + (c & 1) * 8));
        } else {
            const long long j = i - wslabs, t0 = j / p.k64 * 128;
            const int k0 = (int)(j % p.k64) * 64 + c * 8;
            image = ai + j * kImage;
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

// tile index -> (channel pair, token pair): 8 token pairs wide, channel pairs within
__device__ __forceinline__ void tile_at(int i, int cp, int tp, int &c, int &t)
{
    const int band = i / (8 * cp), in = i - band * 8 * cp, wide = min(8, tp - 8 * band);
    c = in / wide;
    t = 8 * band + in - c * wide;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ssd_q8_many_kernel(const Q8Params p, const uint8_t *wi, const uint8_t *ai, int cp, int tp, int ttiles)
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
        if (lane == 0) {
            uint32_t n = 0;   // slabs so far
            bool ok = true;
            for (int i = me; i < items && ok; i += pairs) {
                int c, t;
                tile_at(i, cp, tp, c, t);
                const uint8_t *w = wi + (size_t)min(2 * c + (int)rank, p.tiles - 1) * p.k64 * kImage;
                const uint8_t *a = ai + (size_t)min(2 * t + (int)rank, ttiles - 1) * p.k64 * kImage;
                for (int k = 0; k < p.k64; ++k, ++n) {
                    const uint32_t s = n % kStages;
                    if (n >= kStages && !(ok = wait_bar(&bars[BAR_EMPTY + s], (n / kStages - 1) & 1)))
                        break;
                    mbar_arrive_expect_tx(&bars[BAR_FULL + s], kStageBytes);
                    bulk_load(smem + s * kStageBytes, w + (size_t)k * kImage, kImage, &bars[BAR_FULL + s]);
                    bulk_load(smem + s * kStageBytes + kImage, a + (size_t)k * kImage, kImage, &bars[BAR_FULL + s]);
                }
            }
            // no copy may be under way when shared memory is given up (each stage's last phase)
            for (uint32_t j = n > kStages ? n - kStages : 0; j < n; ++j)
                wait_bar(&bars[BAR_FULL + j % kStages], (j / kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_f16_f32(256, 256);
            uint32_t n = 0, m = 0;   // slabs, accumulators so far
            bool ok = true;
            for (int i = me; i < items && ok; i += pairs)
                for (int ch = 0; ch < chunks && ok; ++ch, ++m) {
                    const uint32_t b = m & 1;
                    if (m >= 2 && !(ok = wait_bar(&bars[BAR_DRAINED + b], (m / 2 - 1) & 1)))
                        break;
                    tc_fence_after();
                    const int end = min(p.k64, (ch + 1) * kChunkSlabs);
                    for (int k = ch * kChunkSlabs; k < end; ++k, ++n) {
                        const uint32_t s = n % kStages;
                        if (!(ok = wait_bar(&bars[BAR_FULL + s], (n / kStages) & 1)))
                            break;
                        tc_fence_after();
                        const uint32_t at = smem_u32(smem + s * kStageBytes);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma2_ss(tmem + 256 * b, sdesc_sw128(at + 32 * kk, 16, 1024), sdesc_sw128(at + kImage + 32 * kk, 16, 1024), idesc,
                                    k > ch * kChunkSlabs || kk > 0);
                        mma2_commit(&bars[BAR_EMPTY + s]);
                    }
                    mma2_commit(&bars[BAR_ACC + b]);
                }
            // no MMA may be in flight when the pair gives its memories up: each accumulator's last
            for (uint32_t j = m > 2 ? m - 2 : 0; j < m; ++j)
                wait_bar(&bars[BAR_ACC + (j & 1)], (j / 2) & 1);
        } else if (lane == 0) {
            // this CTA's copies, told to the leader
            uint32_t n = 0;
            bool ok = true;
            for (int i = me; i < items && ok; i += pairs)
                for (int k = 0; k < p.k64 && ok; ++k, ++n) {
                    if ((ok = wait_bar(&bars[BAR_FULL + n % kStages], (n / kStages) & 1)))
                        mbar_arrive_at(&bars[BAR_FULL + n % kStages], 0);
                }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = warp >> 2;
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128 * half;
        uint32_t m = 0;
        bool ok = true;
        for (int i = me; i < items && ok; i += pairs) {
            int c, t;
            tile_at(i, cp, tp, c, t);
            const int channel = (2 * c + (int)rank) * 128 + 32 * q + lane;
            const long long t0 = 256ll * t + 128 * half;
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
            T *y = static_cast<T *>(p.y) + t0 * p.sy + channel;
            const int left = (int)max(0ll, min(128ll, p.M - t0));
#pragma unroll
            for (int j = 0; j < 128; j += 32) {
                const float as = j + lane < left ? p.as[t0 + j + lane] : 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float f = __shfl_sync(0xffffffffu, as, e);
                    if (mine && j + e < left)
                        y[(j + e) * p.sy] = from_f32<T>((float)acc[j + e] * f * ws);
                }
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
        const int ttiles = (int)((q.M + 127) / 128), cp = (p.tiles + 1) / 2, tp = (ttiles + 1) / 2;
        e = q8_widen_launch(q, ws, ai, m0 == 0 ? wslabs : 0, st);
        if (e != cudaSuccess)
            return e;
        cfg.gridDim = dim3(2 * (unsigned)std::min(cp * tp, sm_count() / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        e = cudaLaunchKernelEx(&cfg, ssd_q8_many_kernel<T>, q, (const uint8_t *)ws, (const uint8_t *)ai, cp, tp, ttiles);
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
    return ((size_t)p.tiles + (size_t)((std::min(kPanel, p.M) + 127) / 128)) * p.k64 * kImage;
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
