// ssd_q8_few.cu -- the 8-bit product for a handful of tokens, bound by the weights' bytes.
//
// One CTA: 16 output channels x up to 8 tokens; its warps take the slabs of 64 inner elements in
// turn and add up their sums at the end.  So there are N / 16 CTAs, several on every SM, without
// an exchange between them (tiles of 128 channels with K split over a cluster: 14.4 us for 8
// tokens of 10576 x 2560, in two uneven waves).  Operands go from memory into registers, 16 bytes
// a lane and row, some slabs at a time, and from there into mma.sync m16n8k32 on 8-bit integers,
// or for one token into dp4a.  sm_103a runs it at 270 products a clock and SM (fp16: 1020), 190 are 8 tokens at the
// memory's rate; widening for the fp16 form took 60 instructions a slab and warp
// and more time than the weights' bytes (10.8 us; with rings of asynchronous copies 13.5).  dp4a has the same
// rate, but no 8 columns to fill: one token takes an eighth of the products (8.4 -> 7.6 us; two already
// take 10.2, 8.8 with mma.sync).  With the prefetch below 1 and 8 tokens of 10576 x 2560 take 6.7 and 8.3 us, 60 and 48%
// of the rate of a plain copy, of 16384 x 8192 28.0 and 32.5 us, 71 and 61%.  At that the products are under half of
// what the tensor cores do; the start and end of each CTA, and the part wave above 12160 channels, are what is
// known of the rest.
// A lane's 16 consecutive elements of a row are two k-steps' fragments when both operands
// are read in the same order, so neither is shuffled.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_internal.h"
#include "ssd_q8.h"

namespace ssd {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kBatch = 5;         // slabs whose loads a warp issues before it uses the first

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void mma16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// TOK: tokens at most; 8 with mma.sync, 1 with dp4a
template <int TOK, typename T>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) ssd_q8_few_kernel(const Q8Params p)
{
    constexpr bool kMma = TOK == 8;
    constexpr int B = kBatch;
    extern __shared__ __align__(16) int part[];   // [warp][token][channel]
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x >> 3, ch0 = (blockIdx.x & 7) * 16;
    // this lane's bytes of a slab's rows g and g + 8 (128 bytes on)
    const int8_t *w = p.w + (size_t)tile * p.k64 * 8192 + t * 2048 + (ch0 + g) * 16;
    // While the launch in front ends: the first weights into L2 (whoever wrote them, it is where they are).
    if (g == 0)
        for (int i = 0; i < B; ++i)
            if (warp + warps * i < p.k64) {
                const int8_t *line = w + (size_t)(warp + warps * i) * 8192;
                asm volatile("prefetch.global.L2 [%0];\n\tprefetch.global.L2 [%0 + 128];" ::"l"(line));
            }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    int sum[kMma ? 4 : 2] = {};   // (dp4a: rows g and g + 8, this lane's elements)
    for (int s = warp; s < p.k64; s += warps * B) {
        uint4 u[B][2], v[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int k = s + warps * i;
            u[i][0] = u[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (k < p.k64) {
                u[i][0] = __ldcs(reinterpret_cast<const uint4 *>(w + (size_t)k * 8192));
                u[i][1] = __ldcs(reinterpret_cast<const uint4 *>(w + (size_t)k * 8192 + 128));
            }
        }
#pragma unroll
        for (int i = 0; i < B; ++i)
            v[i] = load16(p, kMma ? g : 0, (s + warps * i) * 64 + 16 * t);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if constexpr (kMma) {
                mma16832(sum, u[i][0].x, u[i][1].x, u[i][0].y, u[i][1].y, v[i].x, v[i].y);
                mma16832(sum, u[i][0].z, u[i][1].z, u[i][0].w, u[i][1].w, v[i].z, v[i].w);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int &c = sum[h];
                    c = __dp4a((int)u[i][h].x, (int)v[i].x, c);
                    c = __dp4a((int)u[i][h].y, (int)v[i].y, c);
                    c = __dp4a((int)u[i][h].z, (int)v[i].z, c);
                    c = __dp4a((int)u[i][h].w, (int)v[i].w, c);
                }
            }
        }
    }
    if constexpr (kMma) {
#pragma unroll
        for (int e = 0; e < 4; ++e)   // token 2 t + (e & 1), channel g + 8 (e >> 1)
            part[warp * TOK * 16 + (2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = sum[e];
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
            if (t == 0)
                part[warp * 16 + g + 8 * h] = sum[h];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (int)p.M * 16; i += blockDim.x) {
        const int tok = i >> 4, channel = tile * 128 + ch0 + (i & 15);
        if (channel >= p.N)
            continue;
        int v = 0;
        for (int q = 0; q < warps; ++q)
            v += part[q * TOK * 16 + i];
        static_cast<T *>(p.y)[tok * p.sy + channel] = from_f32<T>((float)v * p.as[tok] * p.ws[channel]);
    }
}

template <int TOK, typename T>
cudaError_t launch_t(const Q8Params &p, cudaStream_t st)
{
    // Warps per CTA: as many as let all CTAs run at once with about 20 warps on every SM, as far as that goes: five
    // CTAs of 4 warps are what the registers allow (91 to 93 a thread), 760 in all.  From 12161 channels on
    // some start when others end (12160 and 12176 x 8192: 1 token 18.0 and 21.2 us, 8 tokens 22.0 and 28.0).
    const int items = (p.N + 15) / 16, warps = items <= 2 * sm_count() ? 16 : items <= 3 * sm_count() ? 8 : 4;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(items);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = (size_t)warps * TOK * 16 * 4;
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ssd_q8_few_kernel<TOK, T>, p);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace

cudaError_t q8_few_launch(const Q8Params &p, bool f32, cudaStream_t st)
{
    if (p.M == 1)
        return f32 ? launch_t<1, float>(p, st) : launch_t<1, __nv_bfloat16>(p, st);
    return f32 ? launch_t<8, float>(p, st) : launch_t<8, __nv_bfloat16>(p, st);
}

}  // namespace ssd
