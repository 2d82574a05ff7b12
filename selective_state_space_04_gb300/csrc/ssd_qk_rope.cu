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
//
// Both directions are bound by memory, so what counts is bytes in flight: a warp
// takes a fixed set of heads (a batch: U rows per group of lanes, of one kind,
// so that its weights and gradient sums stay in registers) through tokens in
// steps of the grid, 4 KB a token.  The rows of its next tokens are on their way
// meanwhile, each lane's in a ring of shared-memory slots of its own (16-byte
// asynchronous copies; no slot is shared, so no barrier is needed).  The same
// look-ahead in registers took 180 to 220 of them and ran at half the speed.
// Neighbouring warps take the other heads of the same token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
#ifndef VF
#define VF 4
#define VB 4
#endif
#ifndef VS
#define VS 3
#endif
constexpr int kBlocksPerSm = VF, kBlocksPerSmBwd = VB;   // resident blocks of the forward, of the backward

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

// A lane's slot of one row in shared memory: kChunks pieces of 16 bytes, 512
// bytes apart (the warp's lanes lie side by side).
template <typename T> constexpr int kChunks = sizeof(T) == 2 ? 2 : 4;
template <typename T> constexpr int kRowBytes = kChunks<T> * 512;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ void fetch_slot(uint32_t dst, const T *p, const Slot &t)
{
    constexpr int half = kChunks<T> / 2;
#pragma unroll
    for (int i = 0; i < half; ++i) {
        if (t.a >= 0)
            cp_async16(dst + i * 512, reinterpret_cast<const char *>(p + t.a) + i * 16);
        if (t.b >= 0)
            cp_async16(dst + (half + i) * 512, reinterpret_cast<const char *>(p + t.b) + i * 16);
    }
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// the slot in fp32 (zeros past the head's end)
__device__ __forceinline__ void read_slot(uint32_t a, const Slot &t, float (&x)[8], float (&y)[8], __nv_bfloat16 *)
{
    const uint4 p = t.a >= 0 ? lds16(a) : make_uint4(0, 0, 0, 0), q = t.b >= 0 ? lds16(a + 512) : make_uint4(0, 0, 0, 0);
    const uint32_t u[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        y[2 * i] = __uint_as_float(u[4 + i] << 16);
        y[2 * i + 1] = __uint_as_float(u[4 + i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void read_slot(uint32_t a, const Slot &t, float (&x)[8], float (&y)[8], float *)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 p = t.a >= 0 ? lds16(a + i * 512) : make_uint4(0, 0, 0, 0);
        const uint4 q = t.b >= 0 ? lds16(a + (2 + i) * 512) : make_uint4(0, 0, 0, 0);
        x[4 * i] = __uint_as_float(p.x); x[4 * i + 1] = __uint_as_float(p.y);
        x[4 * i + 2] = __uint_as_float(p.z); x[4 * i + 3] = __uint_as_float(p.w);
        y[4 * i] = __uint_as_float(q.x); y[4 * i + 1] = __uint_as_float(q.y);
        y[4 * i + 2] = __uint_as_float(q.z); y[4 * i + 3] = __uint_as_float(q.w);
    }
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
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = y[j] = 1.f;
    if (w && t.a >= 0)
        load8(w + t.a, x);
    if (w && t.b >= 0)
        load8(w + t.b, y);
}

// the 8 angles of a lane's slot at a position (none for a padding token or an unrotated slot)
__device__ __forceinline__ void load_angles(const QkArgs &a, const Slot &sl, int pos, float (&c)[8], float (&s)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = 1.f;
        s[j] = 0.f;
    }
    if (sl.angle >= 0 && pos >= 0 && pos < a.d.max_pos) {
        const size_t at = (size_t)pos * (a.d.rotary_dim / 2) + sl.angle;
        load8(a.cos + at, c);
        load8(a.sin + at, s);
    }
}

// Rows per group of lanes that a warp has at once: 4 KB a warp.
template <typename T> constexpr int kRowsFwd = sizeof(T) == 2 ? 4 : 2;
template <typename T> constexpr int kRowsBwd = sizeof(T) == 2 ? 2 : 1;

constexpr int kStages = VS;   // tokens in a warp's ring
constexpr int kStageBytes = 4096;

// Batches: the query heads', then the key heads', then (with a cache) the value heads'.
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    ssd_qk_norm_rope_kernel(const __grid_constant__ QkArgs a, int nbq, int nbk, int nb)
{
    constexpr int U = kRowsFwd<T>, G = 32 / LG;
    static_assert(U * kRowBytes<T> == kStageBytes, "a stage");
    extern __shared__ __align__(16) char smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int wid = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int slots = gridDim.x * (kThreads / 32) / nb, batch = wid % nb;
    const int D = a.d.headdim;
    const Slot sl = slot_of(lane % LG, D, a.d.rotary_dim, INTER);
    const int kind = batch < nbq ? 0 : batch < nbq + nbk ? 1 : 2;
    const int H = kind == 0 ? a.d.nheads_q : a.d.nheads_k;
    const int h0 = (batch - (kind == 0 ? 0 : kind == 1 ? nbq : nbq + nbk)) * U * G + lane / LG;   // rows h0, h0 + G, ...
    const int64_t st = kind == 0 ? a.d.q_stride[0] : kind == 1 ? a.d.k_stride[0] : a.d.v_stride[0];
    const int64_t sh = kind == 0 ? a.d.q_stride[1] : kind == 1 ? a.d.k_stride[1] : a.d.v_stride[1];
    const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + h0 * sh;
    T *out = static_cast<T *>(kind == 0 ? a.qo : kind == 1 ? a.ko : nullptr);
    const int64_t ot = kind == 0 ? a.d.qo_stride[0] : a.d.ko_stride[0], oh = kind == 0 ? a.d.qo_stride[1] : a.d.ko_stride[1];
    T *cache = static_cast<T *>(kind == 1 ? a.kc : kind == 2 ? a.vc : nullptr);
    const int64_t *cs = kind == 1 ? a.d.kc_stride : a.d.vc_stride;
    long long t = wid / nb, ahead = t;   // the token at hand, the next to fetch
    if (t >= slots || t >= a.d.ntokens)   // (warps left over from the division into batches)
        return;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * (kStages * kStageBytes) + lane * 16;
    int head = 0, tail = 0;
    auto fetch = [&]() {
        if (ahead < a.d.ntokens) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h0 + u * G < H)
                    fetch_slot(ring + head * kStageBytes + u * kRowBytes<T>, src + ahead * st + u * G * sh, sl);
            ahead += slots;
            head = head + 1 == kStages ? 0 : head + 1;
        }
        cp_commit();
    };
    int pos = a.positions[t];
    long long slot = cache ? a.slots[t] : -1;
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i)
        fetch();
    float wx[8], wy[8];
    load_weight(kind == 0 ? a.qw : a.kw, sl, wx, wy);
    while (true) {
        float c[8], s[8];
        if (kind != 2)
            load_angles(a, sl, pos, c, s);
        const bool pad = pos < 0 || pos >= a.d.max_pos;
        T *dst = out ? out + t * ot : nullptr, *cdst = nullptr;
        if (cache && !pad && slot >= 0) {
            const long long page = slot / a.d.page_size;
            if (page < a.d.npages)
                cdst = cache + page * cs[0] + (slot - page * a.d.page_size) * cs[1];
        }
        t += slots;
        const bool more = t < a.d.ntokens;
        if (more) {
            pos = a.positions[t];
            slot = cache ? a.slots[t] : -1;
        }
        cp_wait<kStages - 2>();   // (a lane reads only what it copied itself)
        const uint32_t stage = ring + tail * kStageBytes;
        tail = tail + 1 == kStages ? 0 : tail + 1;
        if (kind == 2) {   // values are copied as they are
            if (cdst)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h0 + u * G < H) {
                        char *o = reinterpret_cast<char *>(cdst + (long long)(h0 + u * G) * cs[2]);
                        constexpr int half = kChunks<T> / 2;
#pragma unroll
                        for (int i = 0; i < half; ++i) {
                            if (sl.a >= 0)
                                *reinterpret_cast<uint4 *>(o + sl.a * sizeof(T) + i * 16) = lds16(stage + u * kRowBytes<T> + i * 512);
                            if (sl.b >= 0)
                                *reinterpret_cast<uint4 *>(o + sl.b * sizeof(T) + i * 16) =
                                    lds16(stage + u * kRowBytes<T> + (half + i) * 512);
                        }
                    }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * G;
                float x[8], y[8];
                read_slot(stage + u * kRowBytes<T>, sl, x, y, static_cast<T *>(nullptr));
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss += x[j] * x[j] + y[j] * y[j];
                const float r = rsqrtf(group_sum<LG>(ss) / (float)D + a.d.eps);
                if (h < H) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] = pad ? 0.f : x[j] * r * wx[j];
                        y[j] = pad ? 0.f : y[j] * r * wy[j];
                    }
                    if (sl.angle >= 0)
                        rotate<INTER, false>(x, y, c, s);
                    if (dst)
                        store_slot(dst + (long long)h * oh, sl, x, y);
                    if (cdst)
                        store_slot(cdst + (long long)h * cs[2], sl, x, y);
                }
            }
        }
        if (!more)
            break;
        fetch();
    }
    cp_wait<0>();
}

// As the forward's, with the rows' incoming gradients beside them and the
// weights' gradients in registers; a block's are added in a fixed order and leave
// as one row of `part` [blocks][2][D].
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSmBwd)
    ssd_qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a, int nbq, int nb, float *part)
{
    constexpr int U = kRowsBwd<T>, G = 32 / LG, W = kThreads / 32;
    static_assert(2 * U * kRowBytes<T> == kStageBytes, "a stage");
    extern __shared__ __align__(16) char smem[];
    __shared__ float red[W][LG * 16];
    __shared__ int kinds[W];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int w = threadIdx.x >> 5, wid = blockIdx.x * W + w, lane = threadIdx.x & 31;
    const int slots = gridDim.x * W / nb, batch = wid % nb;
    const int D = a.d.headdim;
    const Slot sl = slot_of(lane % LG, D, a.d.rotary_dim, INTER);
    const int kind = batch < nbq ? 0 : 1;
    const int H = kind ? a.d.nheads_k : a.d.nheads_q, h0 = (batch - (kind ? nbq : 0)) * U * G + lane / LG;
    const int64_t xt = kind ? a.d.k_stride[0] : a.d.q_stride[0], xh = kind ? a.d.k_stride[1] : a.d.q_stride[1];
    const int64_t gt = kind ? a.d.ko_stride[0] : a.d.qo_stride[0], gh = kind ? a.d.ko_stride[1] : a.d.qo_stride[1];
    const int64_t dt = kind ? a.d.dk_stride[0] : a.d.dq_stride[0], dh = kind ? a.d.dk_stride[1] : a.d.dq_stride[1];
    const T *xs = static_cast<const T *>(kind ? a.k : a.q) + h0 * xh, *gs = static_cast<const T *>(kind ? a.ko : a.qo) + h0 * gh;
    T *ds = static_cast<T *>(kind ? a.dk : a.dq) + h0 * dh;
    float ax[8], ay[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        ax[j] = ay[j] = 0.f;
    long long t = wid / nb, ahead = t;   // the token at hand, the next to fetch
    const bool works = t < slots && t < a.d.ntokens;
    if (works) {
        const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + w * (kStages * kStageBytes) + lane * 16;
        int head = 0, tail = 0;
        auto fetch = [&]() {
            if (ahead < a.d.ntokens) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h0 + u * G < H) {
                        const uint32_t to = ring + head * kStageBytes + 2 * u * kRowBytes<T>;
                        fetch_slot(to, xs + ahead * xt + u * G * xh, sl);
                        fetch_slot(to + kRowBytes<T>, gs + ahead * gt + u * G * gh, sl);
                    }
                ahead += slots;
                head = head + 1 == kStages ? 0 : head + 1;
            }
            cp_commit();
        };
        int pos = a.positions[t];
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i)
            fetch();
        float wx[8], wy[8];
        load_weight(kind ? a.kw : a.qw, sl, wx, wy);
        while (true) {
            float c[8], s[8];
            load_angles(a, sl, pos, c, s);
            const bool pad = pos < 0 || pos >= a.d.max_pos;
            const long long tok = t;
            t += slots;
            const bool more = t < a.d.ntokens;
            if (more)
                pos = a.positions[t];
            cp_wait<kStages - 2>();
            const uint32_t stage = ring + tail * kStageBytes;
            tail = tail + 1 == kStages ? 0 : tail + 1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], y[8], gx[8], gy[8];
                read_slot(stage + 2 * u * kRowBytes<T>, sl, x, y, static_cast<T *>(nullptr));
                read_slot(stage + (2 * u + 1) * kRowBytes<T>, sl, gx, gy, static_cast<T *>(nullptr));
                if (pad || h0 + u * G >= H) {   // no part in anything, whatever is there
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = y[j] = gx[j] = gy[j] = 0.f;
                }
                if (sl.angle >= 0)
                    rotate<INTER, true>(gx, gy, c, s);
                float ss = 0.f, dot = 0.f;   // sum x^2, sum g w x
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss += x[j] * x[j] + y[j] * y[j];
                    dot += gx[j] * wx[j] * x[j] + gy[j] * wy[j] * y[j];
                }
                ss = group_sum<LG>(ss);
                dot = group_sum<LG>(dot);
                // (with eps 0 the r of a row of zeros would be infinite)
                const float r = ss == 0.f && a.d.eps == 0.f ? 0.f : rsqrtf(ss / (float)D + a.d.eps);
                const float m = r * r * dot / (float)D;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ax[j] += gx[j] * (x[j] * r);
                    ay[j] += gy[j] * (y[j] * r);
                    gx[j] = r * (gx[j] * wx[j] - x[j] * m);
                    gy[j] = r * (gy[j] * wy[j] - y[j] * m);
                }
                if (h0 + u * G < H)
                    store_slot(ds + tok * dt + u * G * dh, sl, gx, gy);
            }
            if (!more)
                break;
            fetch();
        }
        cp_wait<0>();
    }
    if (!part)
        return;
    // the groups of a warp, then the block's warps of either kind
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = 16; o >= LG; o >>= 1) {
            ax[j] += __shfl_xor_sync(0xffffffffu, ax[j], o);
            ay[j] += __shfl_xor_sync(0xffffffffu, ay[j], o);
        }
        if (lane < LG) {
            if (sl.a >= 0)
                red[w][sl.a + j] = ax[j];
            if (sl.b >= 0)
                red[w][sl.b + j] = ay[j];
        }
    }
    if (lane == 0)
        kinds[w] = works ? kind : -1;
    __syncthreads();
    for (int d = threadIdx.x; d < 2 * D; d += kThreads) {
        const int k = d >= D, e = d - k * D;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (kinds[i] == k)
                v += red[i][e];
        part[(size_t)blockIdx.x * 2 * D + d] = v;
    }
}

// dq_weight, dk_weight: the blocks' parts added in a fixed order
__global__ void __launch_bounds__(1024) ssd_qk_weight_grad_kernel(const float *part, float *dqw, float *dkw, int D, int blocks)
{
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// Blocks for `warps` warps of work: as many as run at once, at most.
int blocks_for(long long warps, int per_sm)
{
    const long long b = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return (int)std::min<long long>(std::max<long long>(b, 1), (long long)per_sm * sm_count());
}

int batches(int heads, int rows) { return (heads + rows - 1) / rows; }

constexpr int kRingBytes = kThreads / 32 * kStages * kStageBytes;

template <typename K, typename... A>
cudaError_t launch(K *kernel, int grid, cudaStream_t st, A... args)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int LG>
cudaError_t fwd_lg(const QkArgs &a, cudaStream_t st)
{
    constexpr int rows = kRowsFwd<T> * (32 / LG);
    const int nbq = batches(a.d.nheads_q, rows), nbk = batches(a.d.nheads_k, rows), nb = nbq + nbk * (a.kc ? 2 : 1);
    const int grid = std::max(blocks_for(a.d.ntokens * nb, kBlocksPerSm), batches(nb, kThreads / 32));
    const bool inter = a.d.flags & SSD_ROPE_INTERLEAVED;
    auto kernel = inter ? ssd_qk_norm_rope_kernel<T, LG, true> : ssd_qk_norm_rope_kernel<T, LG, false>;
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = allow_smem(kernel, kRingBytes, done[inter]);
    return e != cudaSuccess ? e : launch(kernel, grid, st, a, nbq, nbk, nb);
}

// batches and blocks of the backward
template <typename T, int LG>
void bwd_sizes(const ssd_qk_dims_t &d, int &nbq, int &nb, int &grid)
{
    constexpr int rows = kRowsBwd<T> * (32 / LG);
    nbq = batches(d.nheads_q, rows);
    nb = nbq + batches(d.nheads_k, rows);
    grid = std::max(blocks_for(d.ntokens * nb, kBlocksPerSmBwd), batches(nb, kThreads / 32));
}

template <typename T, int LG>
cudaError_t bwd_lg(const QkArgs &a, float *part, int *blocks, cudaStream_t st)
{
    int nbq, nb, grid;
    bwd_sizes<T, LG>(a.d, nbq, nb, grid);
    *blocks = grid;
    const bool inter = a.d.flags & SSD_ROPE_INTERLEAVED;
    auto kernel = inter ? ssd_qk_norm_rope_bwd_kernel<T, LG, true> : ssd_qk_norm_rope_bwd_kernel<T, LG, false>;
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = allow_smem(kernel, kRingBytes, done[inter]);
    return e != cudaSuccess ? e : launch(kernel, grid, st, a, nbq, nb, part);
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
cudaError_t bwd_t(const QkArgs &a, float *part, int *blocks, cudaStream_t st)
{
    switch (lanes_for(a.d.headdim)) {
    case 1: return bwd_lg<T, 1>(a, part, blocks, st);
    case 2: return bwd_lg<T, 2>(a, part, blocks, st);
    case 4: return bwd_lg<T, 4>(a, part, blocks, st);
    case 8: return bwd_lg<T, 8>(a, part, blocks, st);
    default: return bwd_lg<T, 16>(a, part, blocks, st);
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
    // one row of the weights' gradients per block
    const int es = d.dtype == SSD_DTYPE_BF16 ? 2 : 4, rows = (es == 2 ? kRowsBwd<__nv_bfloat16> : kRowsBwd<float>) * 32 / lanes_for(d.headdim);
    const int nb = batches(d.nheads_q, rows) + batches(d.nheads_k, rows);
    const int grid = std::max(blocks_for(d.ntokens * nb, kBlocksPerSmBwd), batches(nb, kThreads / 32));
    return d.ntokens > 0 ? (size_t)grid * 2 * d.headdim * sizeof(float) : 0;
}

cudaError_t qk_bwd_launch(const QkArgs &a, void *workspace, cudaStream_t stream)
{
    SSD_NVTX_RANGE("qk_bwd_launch");
    float *part = static_cast<float *>(workspace);
    int blocks = 0;
    cudaError_t e = a.d.dtype == SSD_DTYPE_BF16 ? bwd_t<__nv_bfloat16>(a, part, &blocks, stream)
                                                : bwd_t<float>(a, part, &blocks, stream);
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
                           blocks);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
