// ssd_qk_rope.cu -- per-head RMSNorm of queries and keys with the rotary
// position in the same pass, into the paged cache when serving; and its
// gradients.
//
// A row is one head of one token, D elements.  It is handled by a group of LG
// lanes (LG the power of two >= D / 16), each holding one slot of 2 x 8
// elements in registers: slots below R/16 hold both members of 8 rotated pairs
// (elements 8s.. and R/2 + 8s.. for the half-split form, 16s.. for adjacent
// pairs), so the rotation needs no exchange between lanes, and the pairs'
// angles are cos[8s..8s+7] in both forms; the other slots hold the unrotated
// rest.  The mean square is a sum over the group's lanes by shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;

// 8 consecutive elements in fp32
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// where a lane's slot lies in a row: element offsets of its two chunks of 8
// (-1: none), and the first of its 8 angles (-1: not rotated)
struct Slot {
    int a, b, angle;
};
__device__ __forceinline__ Slot slot_of(int s, int D, int R, bool inter)
{
    Slot t;
    if (s < R / 16) {
        t.a = inter ? 16 * s : 8 * s;
        t.b = inter ? 16 * s + 8 : R / 2 + 8 * s;
        t.angle = 8 * s;
    } else {
        t.a = 16 * s;   // R + 16 (s - R/16)
        t.b = 16 * s + 8;
        t.angle = -1;
        if (t.a >= D)
            t.a = -1;
        if (t.b >= D)
            t.b = -1;
    }
    return t;
}

// (x, y) pairs of the slot: rotated by +angle (fwd) or -angle (bwd)
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float *pa, *pb;
        if (INTER) {   // pair j is elements 2j, 2j + 1 of the slot's 16
            pa = j < 4 ? &x[2 * (j & 3)] : &y[2 * (j & 3)];
            pb = pa + 1;
        } else {
            pa = &x[j];
            pb = &y[j];
        }
        const float a = *pa, b = *pb, sj = BACK ? -s[j] : s[j];
        *pa = a * c[j] - b * sj;
        *pb = b * c[j] + a * sj;
    }
}

template <int LG>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LG / 2; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ void load_slot(const T *p, const Slot &t, float (&x)[8], float (&y)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = y[j] = 0.f;
    if (t.a >= 0)
        load8(p + t.a, x);
    if (t.b >= 0)
        load8(p + t.b, y);
}
template <typename T>
__device__ __forceinline__ void store_slot(T *p, const Slot &t, const float (&x)[8], const float (&y)[8])
{
    if (t.a >= 0)
        store8(p + t.a, x);
    if (t.b >= 0)
        store8(p + t.b, y);
}

__device__ __forceinline__ void load_weight(const float *w, const Slot &t, float (&x)[8], float (&y)[8])
{
    if (w)
        load_slot(w, t, x, y);
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = y[j] = 1.f;
    }
}

// Group g of the grid: token g / gpt, rows g % gpt, + gpt, ... of it.
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads) ssd_qk_norm_rope_kernel(const __grid_constant__ QkArgs a, int gpt)
{
    const int lane = threadIdx.x % LG;
    const long long g = ((long long)blockIdx.x * kThreads + threadIdx.x) / LG;
    const long long t = g / gpt;
    const bool live = t < a.d.ntokens;   // (all lanes stay for the shuffles)
    const int D = a.d.headdim, R = a.d.rotary_dim, Hq = a.d.nheads_q, Hk = a.d.nheads_k;
    const Slot sl = slot_of(lane, D, R, INTER);
    int pos = live ? a.positions[t] : -1;
    const bool pad = pos < 0 || pos >= a.d.max_pos;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = 1.f;
        s[j] = 0.f;
    }
    if (!pad && sl.angle >= 0) {
        load8(a.cos + (size_t)pos * (R / 2) + sl.angle, c);
        load8(a.sin + (size_t)pos * (R / 2) + sl.angle, s);
    }
    long long page = -1;
    int off = 0;
    if (a.kc && live && !pad) {
        const long long slot = a.slots[t];
        if (slot >= 0 && slot / a.d.page_size < a.d.npages) {
            page = slot / a.d.page_size;
            off = (int)(slot - page * a.d.page_size);
        }
    }
    float wx[8], wy[8];
    load_weight(a.qw, sl, wx, wy);
    const int rows = Hq + Hk + (a.kc ? Hk : 0);
    for (int h0 = 0; h0 < rows; h0 += gpt) {   // (uniform trip count: shuffles below)
        const int h = h0 + (int)(g % gpt);
        if (h >= Hq && h - gpt < Hq)
            load_weight(a.kw, sl, wx, wy);
        const bool on = live && h < rows;
        const T *src = nullptr;
        float x[8], y[8];
        if (on) {
            src = h < Hq ? static_cast<const T *>(a.q) + t * a.d.q_stride[0] + (long long)h * a.d.q_stride[1]
                : h < Hq + Hk ? static_cast<const T *>(a.k) + t * a.d.k_stride[0] + (long long)(h - Hq) * a.d.k_stride[1]
                              : static_cast<const T *>(a.v) + t * a.d.v_stride[0] + (long long)(h - Hq - Hk) * a.d.v_stride[1];
            load_slot(src, sl, x, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = y[j] = 0.f;
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss += x[j] * x[j] + y[j] * y[j];
        ss = group_sum<LG>(ss);
        if (!on)
            continue;
        if (h >= Hq + Hk) {   // a value head: copied
            if (page >= 0)
                store_slot(static_cast<T *>(a.vc) + page * a.d.vc_stride[0] + off * a.d.vc_stride[1] +
                               (long long)(h - Hq - Hk) * a.d.vc_stride[2], sl, x, y);
            continue;
        }
        const float r = rsqrtf(ss / (float)D + a.d.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = pad ? 0.f : x[j] * r * wx[j];
            y[j] = pad ? 0.f : y[j] * r * wy[j];
        }
        if (sl.angle >= 0)
            rotate<INTER, false>(x, y, c, s);
        if (h < Hq)
            store_slot(static_cast<T *>(a.qo) + t * a.d.qo_stride[0] + (long long)h * a.d.qo_stride[1], sl, x, y);
        else {
            if (a.ko)
                store_slot(static_cast<T *>(a.ko) + t * a.d.ko_stride[0] + (long long)(h - Hq) * a.d.ko_stride[1], sl, x, y);
            if (page >= 0)
                store_slot(static_cast<T *>(a.kc) + page * a.d.kc_stride[0] + off * a.d.kc_stride[1] +
                               (long long)(h - Hq) * a.d.kc_stride[2], sl, x, y);
        }
    }
}

constexpr int kBwdBlocks = 608;   // 4 blocks per SM; each walks tokens in steps of the grid

// Blocks walk tokens; each group of lanes takes the token's rows gi, gi + gpt, ...
// and keeps its part of the weights' gradients in registers; a block's parts
// are added in a fixed order and leave as one row of `part` [blocks][2][D].
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads) ssd_qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a, float *part)
{
    constexpr int NG = kThreads / LG;
    __shared__ float red[NG][LG * 16 + 4];
    const int lane = threadIdx.x % LG, gi = threadIdx.x / LG;
    const int D = a.d.headdim, R = a.d.rotary_dim;
    const Slot sl = slot_of(lane, D, R, INTER);
    for (int which = 0; which < 2; ++which) {
        const int H = which ? a.d.nheads_k : a.d.nheads_q;
        const T *xs = static_cast<const T *>(which ? a.k : a.q), *gs = static_cast<const T *>(which ? a.ko : a.qo);
        T *ds = static_cast<T *>(which ? a.dk : a.dq);
        const int64_t *xst = which ? a.d.k_stride : a.d.q_stride, *gst = which ? a.d.ko_stride : a.d.qo_stride,
                      *dst = which ? a.d.dk_stride : a.d.dq_stride;
        float wx[8], wy[8], ax[8], ay[8];
        load_weight(which ? a.kw : a.qw, sl, wx, wy);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ax[j] = ay[j] = 0.f;
        for (long long t = blockIdx.x; t < a.d.ntokens; t += gridDim.x) {
            const int pos = a.positions[t];
            const bool pad = pos < 0 || pos >= a.d.max_pos;
            float c[8], s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = 1.f;
                s[j] = 0.f;
            }
            if (!pad && sl.angle >= 0) {
                load8(a.cos + (size_t)pos * (R / 2) + sl.angle, c);
                load8(a.sin + (size_t)pos * (R / 2) + sl.angle, s);
            }
            for (int h0 = 0; h0 < H; h0 += NG) {
                const int h = h0 + gi;
                const bool on = h < H;
                float x[8], y[8], gx[8], gy[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = y[j] = gx[j] = gy[j] = 0.f;
                if (on && !pad) {
                    load_slot(xs + t * xst[0] + (long long)h * xst[1], sl, x, y);
                    load_slot(gs + t * gst[0] + (long long)h * gst[1], sl, gx, gy);
                    if (sl.angle >= 0)
                        rotate<INTER, true>(gx, gy, c, s);
                }
                float ss = 0.f, dot = 0.f;   // sum x^2, sum g w x
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss += x[j] * x[j] + y[j] * y[j];
                    dot += gx[j] * wx[j] * x[j] + gy[j] * wy[j] * y[j];
                }
                ss = group_sum<LG>(ss);
                dot = group_sum<LG>(dot);
                const float r = rsqrtf(ss / (float)D + a.d.eps);
                const float m = r * r * dot / (float)D;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!pad) {
                        ax[j] += gx[j] * (x[j] * r);
                        ay[j] += gy[j] * (y[j] * r);
                    }
                    gx[j] = pad ? 0.f : r * (gx[j] * wx[j] - x[j] * m);
                    gy[j] = pad ? 0.f : r * (gy[j] * wy[j] - y[j] * m);
                }
                if (on)
                    store_slot(ds + t * dst[0] + (long long)h * dst[1], sl, gx, gy);
            }
        }
        if (part) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (sl.a >= 0)
                    red[gi][sl.a + j] = ax[j];
                if (sl.b >= 0)
                    red[gi][sl.b + j] = ay[j];
            }
            __syncthreads();
            for (int d = threadIdx.x; d < D; d += kThreads) {
                float v = 0.f;
                for (int i = 0; i < NG; ++i)
                    v += red[i][d];
                part[((size_t)blockIdx.x * 2 + which) * D + d] = v;
            }
        }
    }
}

// dq_weight, dk_weight: the blocks' parts added in a fixed order
__global__ void __launch_bounds__(1024) ssd_qk_weight_grad_kernel(const float *part, float *dqw, float *dkw, int D, int blocks)
{
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.f;
    if (col < 2 * D)
        for (int b = ty; b < blocks; b += 32)
            v += part[(size_t)b * 2 * D + col];
    red[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && col < 2 * D) {
        float s = 0.f;
        for (int i = 0; i < 32; ++i)
            s += red[i][tx];
        float *out = col < D ? dqw : dkw;
        if (out)
            out[col < D ? col : col - D] = s;
    }
}

// lanes per row: the power of two >= D / 16
int lanes_for(int D)
{
    int lg = 1;
    while (lg * 16 < D)
        lg *= 2;
    return lg;
}

template <typename T, int LG>
cudaError_t fwd_lg(const QkArgs &a, cudaStream_t st)
{
    const int rows = a.d.nheads_q + a.d.nheads_k * (a.kc ? 2 : 1);
    const int gpt = std::min(rows, 8);
    const long long threads = a.d.ntokens * gpt * LG;
    const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
    if (a.d.flags & SSD_ROPE_INTERLEAVED)
        ssd_qk_norm_rope_kernel<T, LG, true><<<grid, kThreads, 0, st>>>(a, gpt);
    else
        ssd_qk_norm_rope_kernel<T, LG, false><<<grid, kThreads, 0, st>>>(a, gpt);
    return cudaGetLastError();
}

int bwd_blocks(const ssd_qk_dims_t &d) { return (int)std::min<int64_t>(kBwdBlocks, std::max<int64_t>(d.ntokens, 1)); }

template <typename T, int LG>
cudaError_t bwd_lg(const QkArgs &a, float *part, cudaStream_t st)
{
    const int grid = bwd_blocks(a.d);
    if (a.d.flags & SSD_ROPE_INTERLEAVED)
        ssd_qk_norm_rope_bwd_kernel<T, LG, true><<<grid, kThreads, 0, st>>>(a, part);
    else
        ssd_qk_norm_rope_bwd_kernel<T, LG, false><<<grid, kThreads, 0, st>>>(a, part);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_t(const QkArgs &a, cudaStream_t st)
{
    switch (lanes_for(a.d.headdim)) {
    case 1: return fwd_lg<T, 1>(a, st);
    case 2: return fwd_lg<T, 2>(a, st);
    case 4: return fwd_lg<T, 4>(a, st);
    case 8: return fwd_lg<T, 8>(a, st);
    default: return fwd_lg<T, 16>(a, st);
    }
}

template <typename T>
cudaError_t bwd_t(const QkArgs &a, float *part, cudaStream_t st)
{
    switch (lanes_for(a.d.headdim)) {
    case 1: return bwd_lg<T, 1>(a, part, st);
    case 2: return bwd_lg<T, 2>(a, part, st);
    case 4: return bwd_lg<T, 4>(a, part, st);
    case 8: return bwd_lg<T, 8>(a, part, st);
    default: return bwd_lg<T, 16>(a, part, st);
    }
}

}  // namespace

cudaError_t qk_fwd_launch(const QkArgs &a, cudaStream_t stream)
{
    SSD_NVTX_RANGE("qk_fwd_launch");
    const cudaError_t e = a.d.dtype == SSD_DTYPE_BF16 ? fwd_t<__nv_bfloat16>(a, stream) : fwd_t<float>(a, stream);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

size_t qk_bwd_workspace_bytes(const ssd_qk_dims_t &d)
{
    return d.ntokens > 0 ? (size_t)bwd_blocks(d) * 2 * d.headdim * sizeof(float) : 0;
}

cudaError_t qk_bwd_launch(const QkArgs &a, void *workspace, cudaStream_t stream)
{
    SSD_NVTX_RANGE("qk_bwd_launch");
    float *part = static_cast<float *>(workspace);
    cudaError_t e = a.d.dtype == SSD_DTYPE_BF16 ? bwd_t<__nv_bfloat16>(a, part, stream) : bwd_t<float>(a, part, stream);
    if (e != cudaSuccess)
        return e;
    note_launches(1);
    if (!part)
        return cudaSuccess;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * a.d.headdim + 31) / 32));
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, ssd_qk_weight_grad_kernel, (const float *)part, a.dqw, a.dkw, (int)a.d.headdim,
                           bwd_blocks(a.d));
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
