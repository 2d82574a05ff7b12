// ssd_q8_mid.cu -- the 8-bit product for up to a few hundred tokens, on tcgen05.
//
// One CTA: 128 output channels x up to 128 tokens x a range of K, in slabs of 64 inner
// elements.  sm_103a's tensor cores take 8-bit integers slowly, so both operands are widened to
// fp16, which holds -128 .. 127 exactly, and the products are added in fp32: exactly, as
// long as a partial sum stays below 2^24, which 1024 products of at most 2^14 do.
// So every 1024 inner elements have an accumulator of their own, as far as TMEM goes;
// beyond that the accumulators are drained into 32-bit integers in shared memory.
//
// A slab's weights (8 KB, contiguous) come by bulk copy; two groups of four warps take the
// slabs in turn, widen them, a thread per channel, and put them into TMEM as the MMA's A
// operand, which keeps them out of shared memory's bandwidth: at the memory's rate the
// weights alone would take 6.8 TB/s into shared memory, as much out, and twice that again
// each way as fp16.  The tokens, the B operand, are widened by a small launch in
// front, into the images that the copies bring (ssd_q8_many.cu): widened in here, the
// fence between ordinary stores and the MMA waits for every load under way as well,
// which cost a memory latency a slab (128 tokens: 23.7 us).
//
// K is split over a cluster of CTAs where there are few tiles; each CTA ends with the
// sums of its range, they are exchanged through distributed shared memory, every CTA
// adding and storing its part of the tokens.  Sums are integers: any order is exact.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "ssd_internal.h"
#include "ssd_q8.h"

namespace ssd {

using namespace ptx;

static __device__ unsigned int g_q8_mid_error;

namespace {

constexpr int kThreads = 352;   // warps 0-7: weights and results, 8: copies of weights, 9: MMA, 10: copies of tokens
constexpr int kSlabBytes = 128 * 64;
constexpr int kChunkSlabs = 16;   // slabs of one accumulator: 1024 inner elements
constexpr uint64_t kTimeoutNs = 2000000000ull;

// kAlone: one CTA on an SM, K not split: all of TMEM, rings twice as deep (a slab's way from L2 takes three
// times as long as its MMAs), drained sums in registers.  Else two CTAs on an SM, K split over
// a cluster where there are few tiles, drained sums in shared memory where there are any.
template <int MT, bool kAlone> struct Shape {
    // Weight slabs on their way.  With them a CTA that shares an SM takes more than a third of its shared
    // memory: a third CTA on the SM would wait for tensor memory, and the CTAs of two clusters
    // that wait for each other's that way would wait for ever.
    // Even, as kStages is: a place in either ring then always has the same group of warps, which has
    // seen each of its phases (a wait for a phase whose predecessor is not done with passes).
    static constexpr int kW = MT == 128 && !kAlone ? 4 : 8;
    static constexpr int kStages = kAlone ? 8 : 4;        // slabs in TMEM (A) and shared memory (B)
    static_assert(kW % 2 == 0 && kStages % 2 == 0, "two groups take the slabs in turn");
    static constexpr int kB = MT * 128;                   // a slab of tokens as fp16
    static constexpr int kOffB = 0;                       // (1024-byte aligned)
    static constexpr int kOffW = kStages * kB;
    static constexpr int kRings = kOffW + kW * kSlabBytes;
    static constexpr int kSums = 128 * MT * 4;            // drained sums, [token][channel]
    // TMEM: accumulators, then the weights' stages
    static constexpr int kCols = kAlone ? 512 : 256, kColA = kCols - 32 * kStages;
    static constexpr int kAccs = kColA / MT;
    static constexpr int kRound = kAccs * kChunkSlabs;    // slabs between drains
    static_assert(kRings > 78 * 1024, "three CTAs would fit");
    static_assert(kRings >= (MT + 7 * 8) * 128 * 4, "the exchange takes the rings' place");
    static_assert(kRound % kW == 0 && kChunkSlabs % kStages == 0, "a round ends with a turn of the rings");
    enum { BAR_WFULL, BAR_WEMPTY = kW, BAR_A = 2 * kW, BAR_B = BAR_A + kStages, BAR_EMPTY = BAR_B + kStages, BAR_ACC = BAR_EMPTY + kStages, BAR_DRAINED,
           kBars };
};


__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_test(bar, parity))
                return true;
    } while (globaltimer_ns() - t0 < kTimeoutNs);
    atomicCAS(&g_q8_mid_error, 0u, (unsigned)SSD_ERR_TIMEOUT);
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
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <int MT, bool kAlone, typename T>
__global__ void __launch_bounds__(kThreads, kAlone ? 1 : 2) ssd_q8_mid_kernel(const Q8Params p, const uint8_t *images, int splits, int multi)
{
    using S = Shape<MT, kAlone>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[S::kBars];
    __shared__ uint32_t holder;
    __shared__ float token_scale[MT];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / splits, rank = blockIdx.x - tile * splits;
    const long long t0 = (long long)blockIdx.y * MT;
    // this CTA's slabs
    const int first = (int)((long long)p.k64 * rank / splits), last = (int)((long long)p.k64 * (rank + 1) / splits);
    const int slabs = last - first;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kW; ++i) {
            mbar_init(&bars[S::BAR_WFULL + i], 1);
            mbar_init(&bars[S::BAR_WEMPTY + i], 4);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars[S::BAR_A + i], 4);
            mbar_init(&bars[S::BAR_B + i], 1);
            mbar_init(&bars[S::BAR_EMPTY + i], 1);
        }
        mbar_init(&bars[S::BAR_ACC], 1);
        mbar_init(&bars[S::BAR_DRAINED], 8);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&holder, S::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = holder;
    // The launch in front of this one writes the tokens' images, and has waited for all before it before
    // it let this one begin: weights and scales may be read at once, the images after the wait.  From L2, where
    // the launches before that one have left them; what this SM's L1 holds is settled by the wait only.
    bool ok = true;
    for (int i = threadIdx.x; i < MT; i += kThreads)
        token_scale[i] = t0 + i < p.M ? __ldcg(p.as + t0 + i) : 0.f;

    const int n = threadIdx.x & 127;   // (of warps 0-7: their channel)
    const bool mine = tile * 128 + n < p.N;
    const float ws = warp < 8 && mine ? __ldcg(p.ws + tile * 128 + n) : 0.f;
    const uint32_t quarter = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    int *sums = reinterpret_cast<int *>(smem + S::kRings) + 32 * (warp & 3) + lane;   // (with `multi`, not alone)
    int kept[kAlone ? MT / 2 : 1] = {};                                               // (alone: every other 8 tokens)
    // warps 0-7: 8 tokens' sums of the accumulators in use, and of what was drained before
    auto collect = [&](int c0, int accs, bool more, int (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = more ? sums[(c0 + i) * 128] : 0;
        for (int j = 0; j < accs; ++j) {
            uint32_t u[8];
            tmem_ld8(quarter + j * MT + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += __float2int_rn(__uint_as_float(u[i]));
        }
    };

    if (warp < 8) {
        const int row = 32 * (warp & 3) + lane, group = warp >> 2;
        for (int round = 0, k = group; ok; ++round) {
            const int end = min(slabs, (round + 1) * S::kRound);
            for (; k < end && ok; k += S::kW) {
                const uint32_t wpar = (k / S::kW) & 1;
#pragma unroll
                for (int i = 0; i < S::kW; i += 2) {
                    if (k + i >= end)
                        break;
                    const int w = i + group, s = w % S::kStages;
                    const uint32_t spar = ((k + i) / S::kStages - 1) & 1;
                    if (!(ok = warp_wait(&bars[S::BAR_WFULL + w], wpar)))
                        break;
                    uint32_t f[32];
                    const uint8_t *src = smem + S::kOffW + w * kSlabBytes + row * 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        widen16(*reinterpret_cast<const uint4 *>(src + c * 2048), &f[8 * c]);
                    warp_arrive(&bars[S::BAR_WEMPTY + w]);
                    if (k + i >= S::kStages && !(ok = warp_wait(&bars[S::BAR_EMPTY + s], spar)))
                        break;
                    tc_fence_after();
                    tmem_st32(quarter + S::kColA + 32 * s, f);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bars[S::BAR_A + s]);
                }
            }
            if (!ok || !(ok = warp_wait(&bars[S::BAR_ACC], round & 1)))
                break;
            tc_fence_after();
            if (end == slabs)
                break;
            if constexpr (kAlone) {
#pragma unroll
                for (int c = 0; c < MT / 2; c += 8) {
                    int v[8];
                    collect(2 * c + 8 * group, S::kAccs, false, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        kept[c + i] += v[i];
                }
            } else {
                for (int c0 = 8 * group; c0 < MT; c0 += 16) {   // (only with `multi`)
                    int v[8];
                    collect(c0, S::kAccs, round > 0, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sums[(c0 + i) * 128] = v[i];
                }
            }
            tc_fence_before();
            warp_arrive(&bars[S::BAR_DRAINED]);
        }
    } else if (warp == 8 || warp == 10) {
        // slabs of weights or tokens into their rings
        const bool issue = elect_one(), weights = warp == 8;
        const size_t step = weights ? (size_t)kSlabBytes : (size_t)p.padded() * 128;
        const uint8_t *src = weights ? reinterpret_cast<const uint8_t *>(p.w) + ((size_t)tile * p.k64 + first) * kSlabBytes
                                     : images + first * step + t0 * 128;
        const int places = weights ? S::kW : S::kStages, bytes = weights ? kSlabBytes : S::kB;
        uint64_t *full = &bars[weights ? S::BAR_WFULL : S::BAR_B], *empty = &bars[weights ? S::BAR_WEMPTY : S::BAR_EMPTY];
        uint8_t *ring = smem + (weights ? S::kOffW : S::kOffB);
        if (!weights)
            asm volatile("griddepcontrol.wait;" ::: "memory");
        int k = 0, at = 0;
        uint32_t parity = 1;   // (of the places' last uses)
        for (; k < slabs; ++k, src += step) {
            if (k >= places && !(ok = warp_wait(&empty[at], parity)))
                break;
            if (issue) {
                mbar_arrive_expect_tx(&full[at], bytes);
                bulk_load(ring + at * bytes, src, bytes, &full[at]);
            }
            __syncwarp();
            if (++at == places) {
                at = 0;
                parity ^= 1;
            }
        }
        // no copy may be under way when shared memory is given up
        for (int j = max(0, k - places); j < k; ++j)
            wait_bar(&full[j % places], (j / places) & 1);
        __syncwarp();
    } else {
        {   // (warp 9)
            const bool issue = elect_one();
            constexpr uint32_t idesc = idesc_f16_f32(128, MT);
            const uint64_t b0 = sdesc_sw128(smem_u32(smem + S::kOffB), 16, 1024);
            uint32_t round = 0, parity = 0;
            // one warp walks this, and its instructions are what a slab takes at least: stages and descriptors
            // are constants, the rest is looked at once a turn of the rings
            for (int k = 0; k < slabs && ok; k += S::kStages, parity ^= 1) {
                if (k > 0 && k % S::kRound == 0) {
                    if (issue)
                        mma_commit(&bars[S::BAR_ACC]);
                    __syncwarp();
                    if (!(ok = warp_wait(&bars[S::BAR_DRAINED], round & 1)))
                        break;
                    tc_fence_after();
                    ++round;
                }
                const uint32_t acc = tmem + (k / kChunkSlabs) % S::kAccs * MT;
                const uint32_t more = k % kChunkSlabs > 0;
#pragma unroll
                for (int s = 0; s < S::kStages; ++s) {
                    if (k + s >= slabs)
                        break;
                    if (!(ok = warp_wait(&bars[S::BAR_A + s], parity) && warp_wait(&bars[S::BAR_B + s], parity)))
                        break;
                    tc_fence_after();
                    if (issue) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // (descriptors count 16 bytes)
                            mma_ts(acc, tmem + S::kColA + 32 * s + 8 * kk, b0 + (s * S::kB + 32 * kk) / 16, idesc, s + kk > 0 ? 1u : more);
                        mma_commit(&bars[S::BAR_EMPTY + s]);
                    }
                    __syncwarp();
                }
            }
            if (issue)
                mma_commit(&bars[S::BAR_ACC]);   // (every MMA issued so far)
            __syncwarp();
            warp_wait(&bars[S::BAR_ACC], round & 1);
        }
        __syncwarp();
    }
    // (whoever is launched after this one waits for its end before it touches anything)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int accs = ((slabs - 1) % S::kRound) / kChunkSlabs + 1;
    const bool more = multi && slabs > S::kRound;
    T *y = static_cast<T *>(p.y) + t0 * p.sy + tile * 128;
    const int left = (int)min((long long)MT, p.M - t0);   // tokens
    if (kAlone || splits == 1) {
        __syncthreads();   // (token_scale)
        if (warp < 8 && ok)
#pragma unroll
            for (int c = 0; c < MT / 2; c += 8) {
                const int c0 = 2 * c + 8 * (warp >> 2);
                if (c0 >= left)
                    break;
                int v[8];
                collect(c0, accs, more && !kAlone, v);
                T *to = y + c0 * p.sy + n;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (kAlone)
                        v[i] += kept[kAlone ? c + i : 0];
                    if (mine && c0 + i < left)
                        to[i * p.sy] = from_f32<T>((float)v[i] * token_scale[c0 + i] * ws);
                }
            }
    } else {
        // CTA q of the cluster adds up and stores the tokens q * cols ...: the others put their sums of
        // these into its shared memory, where the rings were; they are done with in this CTA
        // (the last wait above was for every MMA) and, after the barrier, in the whole cluster.
        // The sums of 4 tokens lie side by side, [4 tokens][channel][token], so that both the
        // stores to the other SMs and the loads are 16 bytes a lane.
        const int cols = ((MT + splits - 1) / splits + 7) / 8 * 8;
        cluster_sync();
        if (warp < 8 && ok)
            for (int c0 = 8 * (warp >> 2); c0 < left; c0 += 16) {
                int v[8];
                collect(c0, accs, more, v);
                const int owner = c0 / cols;
                const uint32_t to = cluster_addr(smem_u32(smem) + 16u * ((rank * cols + c0 - owner * cols) / 4 * 128 + n), owner);
                cluster_st4(to, v[0], v[1], v[2], v[3]);
                cluster_st4(to + 2048u, v[4], v[5], v[6], v[7]);
            }
        cluster_sync();
        const int c1 = min(cols, left - rank * cols);
        const int4 *parts = reinterpret_cast<const int4 *>(smem) + n;
        if (warp < 8 && mine)
#pragma unroll 2
            for (int c = 4 * (warp >> 2); c < c1; c += 8) {
                int4 v = make_int4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < splits) {
                        const int4 u = parts[(q * cols + c) / 4 * 128];
                        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
                    }
                const int w[4] = {v.x, v.y, v.z, v.w};
                T *to = y + (rank * cols + c) * p.sy + n;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < c1)
                        to[i * p.sy] = from_f32<T>((float)w[i] * token_scale[rank * cols + c + i] * ws);
            }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
}

template <int MT, bool kAlone, typename T>
cudaError_t launch_t(const Q8Params &p, const uint8_t *images, int splits, cudaStream_t st)
{
    using S = Shape<MT, kAlone>;
    const int most = (p.k64 + splits - 1) / splits;
    const int multi = !kAlone && most > S::kRound;
    const int smem = S::kRings + (multi ? S::kSums : 0) + 1024;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(ssd_q8_mid_kernel<MT, kAlone, T>, S::kRings + (kAlone ? 0 : S::kSums) + 1024, done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.tiles * splits, (unsigned)((p.M + MT - 1) / MT));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (kAlone) {
        at[0] = at[1];
        cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelEx(&cfg, ssd_q8_mid_kernel<MT, kAlone, T>, p, images, splits, multi);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

// splits 0: CTAs alone on their SMs
template <typename T>
cudaError_t launch_mt(const Q8Params &p, const uint8_t *images, int mt, int splits, cudaStream_t st)
{
    if (splits == 0)
        return mt == 32   ? launch_t<32, true, T>(p, images, 1, st)
               : mt == 64 ? launch_t<64, true, T>(p, images, 1, st)
                          : launch_t<128, true, T>(p, images, 1, st);
    return mt == 32   ? launch_t<32, false, T>(p, images, splits, st)
           : mt == 64 ? launch_t<64, false, T>(p, images, splits, st)
                      : launch_t<128, false, T>(p, images, splits, st);
}

}  // namespace

size_t q8_mid_workspace_bytes(const Q8Params &p) { return (size_t)p.padded() * p.k64 * 128; }

cudaError_t q8_mid_launch(const Q8Params &p, bool f32, void *workspace, cudaStream_t st)
{
    const int mt = p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
    const long long tiles = (long long)p.tiles * ((p.M + mt - 1) / mt);
    // What a call takes by measurement, in 10 ns.  A CTA alone on its SM: 23.5 a slab and 150 + 3.7 a token for its
    // start and results (128 tokens, with the launch in front: 18.7 us for 10576 x 2560, 37 for 500 x 8000, 40
    // for 16384 x 8192).  With K in ranges and the exchange between them: 25 a slab and 300 + 3 a token, and
    // where two share an SM 32 each and 400 + 4 a token (17.3, 11.9 and 60 us).  Clusters of more than two leave
    // some SMs' second place empty (of 304 places 291 to 296 are taken up to four, 266 to 290 up to eight).
    // (235 ns are about 480 clocks; the MMAs of a slab and 128 tokens take 259, and two CTAs that share an SM 320 ns for
    // two slabs.  What the others of a CTA alone go to was not isolated.)
    const long long sms = sm_count(), round = 128 / mt * kChunkSlabs;
    auto waves = [](long long n, long long at_once) { return (n + at_once - 1) / at_once; };
    long long best = waves(tiles, sms) * (p.k64 * 47 / 2 + 150 + mt * 37 / 10 + (p.k64 - 1) / (2 * round) * 100);
    int splits = 0;   // (alone)
    for (int n : {1, 2, 3, 4, 6, 8}) {   // (five and seven place worse still)
        if (n > 1 && 2 * n > p.k64)
            break;
        const long long slabs = (p.k64 + n - 1) / n;
        const bool apart = tiles * n <= sms || slabs > round;   // (drained sums take the second CTA's place)
        const long long at_once = apart ? sms : n > 4 ? 2 * sms * 7 / 8 : n > 2 ? 2 * sms * 15 / 16 : 2 * sms;
        const long long ends = n == 1 ? 150 + mt * 37 / 10 : apart ? 300 + mt * 3 : 400 + mt * 4;
        const long long cost = waves(tiles * n, at_once) * (slabs * (apart ? 25 : 32) + ends + (slabs - 1) / round * 150);
        if (cost < best) {
            best = cost;
            splits = n;
        }
    }
    uint8_t *images = static_cast<uint8_t *>(workspace);
    const cudaError_t e = q8_widen_launch(p, nullptr, images, 0, st);
    if (e != cudaSuccess)
        return e;
    if (f32)
        return launch_mt<float>(p, images, mt, splits, st);
    return launch_mt<__nv_bfloat16>(p, images, mt, splits, st);
}

ssd_status_t q8_mid_read_device_error(uint32_t *code)
{
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_q8_mid_error, sizeof(v)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_q8_mid_error, &zero, sizeof(zero)) != cudaSuccess)
        return SSD_ERR_CUDA;
    *code = v;
    return SSD_OK;
}

}  // namespace ssd
