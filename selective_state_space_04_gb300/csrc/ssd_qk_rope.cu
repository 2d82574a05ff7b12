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
// rest.  The mean square is a sum over the group's lanes by shuffles; the
// arithmetic is packed pairs of fp32.
//
// Both directions are bound by memory, so what counts is bytes in flight, and
// for those resident warps, and for those registers.  The rows of all tokens and
// heads of one kind (queries, keys, values) lie end to end, and a block takes
// consecutive ones of one kind, whatever the number of heads: strides and
// weights are then the same for the whole block.  Rows are read and written past
// the caches' usual order (streaming: 145 -> 136 us forward).  Tried and slower:
// the next rows on their way in registers (178 us at best) or in per-lane rings of
// shared memory (152), weights and angles read anew for every row (151): what
// limits is instructions and L1 traffic beside the rows' own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "f32x2.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
// Resident blocks that the registers leave room for, and rows per group of lanes
// at once.  Measured on 32768 tokens of 32 + 8 heads of 128 (bf16, into the
// cache; backward): 6 blocks of 2 rows 136 us, 4 of 4 rows 150, 8 of 2 rows (spills)
// 152; backward 4 blocks of 2 rows 174 us, 3 of 2 rows 191, 4 of 1 row 196.
constexpr int kFwdPerSm = 6, kBwdPerSm = 4;

template <typename T> constexpr int kRowsFwd = sizeof(T) == 2 ? 2 : 1;
template <typename T> constexpr int kRowsBwd = sizeof(T) == 2 ? 2 : 1;

// exact floor(n / d) for 0 <= n < 2^31: (n * mul) >> sh
struct FastDiv {
    uint32_t mul, sh;
    int d;
    explicit FastDiv(int n = 1) : sh(31), d(n)
    {
        while ((1u << (sh - 31)) < (uint32_t)n)
            ++sh;
        mul = (uint32_t)((1ull << sh) / (uint32_t)n + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> sh); }
};

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

// A lane's slot of a row as it lies in memory.
template <typename T> struct Raw {
    static constexpr int kHalf = (int)sizeof(T) / 2;   // 16-byte pieces of 8 elements
    uint4 a[kHalf], b[kHalf];
    __device__ __forceinline__ void load(const T *p, const Slot &t, bool on)
    {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            a[i] = on && t.a >= 0 ? __ldcs(reinterpret_cast<const uint4 *>(p + t.a) + i) : make_uint4(0, 0, 0, 0);
            b[i] = on && t.b >= 0 ? __ldcs(reinterpret_cast<const uint4 *>(p + t.b) + i) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void store(T *p, const Slot &t) const
    {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            if (t.a >= 0)
                __stcs(reinterpret_cast<uint4 *>(p + t.a) + i, a[i]);
            if (t.b >= 0)
                __stcs(reinterpret_cast<uint4 *>(p + t.b) + i, b[i]);
        }
    }
    __device__ __forceinline__ static void pairs(const uint4 (&v)[kHalf], f32x2 (&f)[4])
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = pk2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[2 * i] = pk2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                f[2 * i + 1] = pk2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        }
    }
    __device__ __forceinline__ void get(f32x2 (&x)[4], f32x2 (&y)[4]) const
    {
        pairs(a, x);
        pairs(b, y);
    }
    __device__ __forceinline__ static void pack(const f32x2 (&f)[4], uint4 (&v)[kHalf])
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(lo2(f[i]), hi2(f[i]));
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = make_uint4(__float_as_uint(lo2(f[2 * i])), __float_as_uint(hi2(f[2 * i])),
                                  __float_as_uint(lo2(f[2 * i + 1])), __float_as_uint(hi2(f[2 * i + 1])));
        }
    }
    __device__ __forceinline__ void set(const f32x2 (&x)[4], const f32x2 (&y)[4])
    {
        pack(x, a);
        pack(y, b);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
            a[i] = b[i] = make_uint4(0, 0, 0, 0);
    }
};

// 8 consecutive fp32 as pairs
__device__ __forceinline__ void load_pairs(const float *p, f32x2 (&f)[4])
{
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

__device__ __forceinline__ f32x2 swap2(f32x2 v) { return pk2(hi2(v), lo2(v)); }
__device__ __forceinline__ f32x2 neg2(f32x2 v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ float sum2(f32x2 v) { return lo2(v) + hi2(v); }

// rotates the slot's elements by the angle (BACK: by minus the angle) of each of its 8 pairs
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate(f32x2 (&x)[4], f32x2 (&y)[4], const f32x2 (&c)[4], const f32x2 (&s)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!INTER) {   // x[j], y[j] are a pair
            const f32x2 a = x[i], b = y[i];
            x[i] = fma2(a, c[i], mul2(b, BACK ? s[i] : neg2(s[i])));
            y[i] = fma2(b, c[i], mul2(a, BACK ? neg2(s[i]) : s[i]));
        } else {        // elements 2i, 2i + 1 of x are pair i, of y pair 4 + i
            const f32x2 cx = c[i >> 1], sx = s[i >> 1], cy = c[2 + (i >> 1)], sy = s[2 + (i >> 1)];
            const float c0 = i & 1 ? hi2(cx) : lo2(cx), s0 = i & 1 ? hi2(sx) : lo2(sx);
            const float c1 = i & 1 ? hi2(cy) : lo2(cy), s1 = i & 1 ? hi2(sy) : lo2(sy);
            x[i] = fma2(x[i], pk2(c0, c0), mul2(swap2(x[i]), BACK ? pk2(s0, -s0) : pk2(-s0, s0)));
            y[i] = fma2(y[i], pk2(c1, c1), mul2(swap2(y[i]), BACK ? pk2(s1, -s1) : pk2(-s1, s1)));
        }
    }
}

// the weights of the slot's elements (1 without weights)
__device__ __forceinline__ void load_weight(const float *w, const Slot &t, f32x2 (&x)[4], f32x2 (&y)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = y[i] = pk2(1.f, 1.f);
    if (w && t.a >= 0)
        load_pairs(w + t.a, x);
    if (w && t.b >= 0)
        load_pairs(w + t.b, y);
}

// cos and sin of the slot's 8 pairs at a position (of a padding token, or an unrotated slot: not read)
__device__ __forceinline__ void load_angles(const QkArgs &a, const Slot &t, int pos, f32x2 (&c)[4], f32x2 (&s)[4])
{
    if (t.angle >= 0 && pos >= 0 && pos < a.d.max_pos) {
        const size_t at = (size_t)pos * (a.d.rotary_dim / 2) + t.angle;
        load_pairs(a.cos + at, c);
        load_pairs(a.sin + at, s);
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

// Blocks of the kinds of rows: queries', then keys', then (forward, with a cache)
// values'.
struct RowGrid {
    FastDiv hq, hk;
    int q, k, v;   // blocks of either kind
    float inv_d;
};

// A warp takes U * G consecutive rows of its block's kind at a time (2 KB of
// heads of 128), group gi of it rows gi, G + gi, ..., all of them loaded first; the
// angles are loaded again only where the token changes.
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads, kFwdPerSm)
    ssd_qk_norm_rope_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ RowGrid g)
{
    constexpr int U = kRowsFwd<T>, G = 32 / LG;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int block = blockIdx.x, kind = block < g.q ? 0 : block < g.q + g.k ? 1 : 2;
    const int first = ((block - (kind == 0 ? 0 : kind == 1 ? g.q : g.q + g.k)) * (kThreads / 32) + (threadIdx.x >> 5)) * (U * G) +
                      (threadIdx.x & 31) / LG;
    const FastDiv &by = kind == 0 ? g.hq : g.hk;
    const int n = (int)a.d.ntokens * by.d, D = a.d.headdim;
    const Slot sl = slot_of(threadIdx.x % LG, D, a.d.rotary_dim, INTER);
    const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
    const int64_t *ss = kind == 0 ? a.d.q_stride : kind == 1 ? a.d.k_stride : a.d.v_stride;
    int tok[U], pos[U];
    Raw<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = first + u * G;
        tok[u] = by(min(row, n - 1));
        pos[u] = a.positions[tok[u]];
        raw[u].load(src + tok[u] * ss[0] + (row - tok[u] * by.d) * ss[1], sl, row < n);
    }
    T *out = static_cast<T *>(kind == 0 ? a.qo : kind == 1 ? a.ko : nullptr);
    const int64_t *os = kind == 0 ? a.d.qo_stride : a.d.ko_stride;
    T *cache = static_cast<T *>(kind == 1 ? a.kc : kind == 2 ? a.vc : nullptr);
    const int64_t *cs = kind == 1 ? a.d.kc_stride : a.d.vc_stride;
    f32x2 wx[4], wy[4], c[4], s[4];
    if (kind < 2)
        load_weight(kind == 0 ? a.qw : a.kw, sl, wx, wy);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = first + u * G, h = row - tok[u] * by.d;
        const bool on = row < n, pad = pos[u] < 0 || pos[u] >= a.d.max_pos;
        if (kind < 2) {   // (values are copied as they are)
            f32x2 x[4], y[4], sq = pk2(0.f, 0.f);
            if (u == 0 || tok[u] != tok[u > 0 ? u - 1 : 0])
                load_angles(a, sl, pos[u], c, s);
            raw[u].get(x, y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sq = fma2(y[i], y[i], fma2(x[i], x[i], sq));
            const float r = rsqrtf(group_sum<LG>(sum2(sq)) * g.inv_d + a.d.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = mul2(mul2(x[i], pk2(r, r)), wx[i]);
                y[i] = mul2(mul2(y[i], pk2(r, r)), wy[i]);
            }
            if (sl.angle >= 0 && !pad)
                rotate<INTER, false>(x, y, c, s);
            raw[u].set(x, y);
            if (pad)
                raw[u].clear();
            if (out && on)
                raw[u].store(out + tok[u] * os[0] + h * os[1], sl);
        }
        if (cache && on && !pad) {
            const long long slot = a.slots[tok[u]], page = slot / a.d.page_size;
            if (slot >= 0 && page < a.d.npages)
                raw[u].store(cache + page * cs[0] + (slot - page * a.d.page_size) * cs[1] + h * cs[2], sl);
        }
    }
}

// The weights' gradients stay in registers; a block's are added in a fixed order
// and leave as one row of `part` [blocks][D].
template <typename T, int LG, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdPerSm)
    ssd_qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ RowGrid g, float *part)
{
    constexpr int U = kRowsBwd<T>, G = 32 / LG, W = kThreads / 32;
    __shared__ float red[W][LG * 16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool key = (int)blockIdx.x >= g.q;
    const FastDiv &by = key ? g.hk : g.hq;
    const int n = (int)a.d.ntokens * by.d, D = a.d.headdim, step = (key ? g.k : g.q) * (W * U * G);
    const Slot sl = slot_of(threadIdx.x % LG, D, a.d.rotary_dim, INTER);
    const T *xs = static_cast<const T *>(key ? a.k : a.q), *gs = static_cast<const T *>(key ? a.ko : a.qo);
    T *ds = static_cast<T *>(key ? a.dk : a.dq);
    const int64_t *xst = key ? a.d.k_stride : a.d.q_stride, *gst = key ? a.d.ko_stride : a.d.qo_stride,
                  *dst = key ? a.d.dk_stride : a.d.dq_stride;
    f32x2 ax[4], ay[4], wx[4], wy[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ax[i] = ay[i] = pk2(0.f, 0.f);
    load_weight(key ? a.kw : a.qw, sl, wx, wy);
    // (the warp's first row decides, so that its lanes stay together for the shuffles)
    const int gi = (threadIdx.x & 31) / LG;
    for (int base = ((blockIdx.x - (key ? g.q : 0)) * W + (threadIdx.x >> 5)) * (U * G); base < n; base += step) {
        int tok[U], pos[U];
        Raw<T> rx[U], rg[U];
        f32x2 c[4], s[4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = base + u * G + gi;
            const bool on = row < n;
            tok[u] = by(on ? row : n - 1);
            const int h = row - tok[u] * by.d;
            pos[u] = a.positions[tok[u]];
            rx[u].load(xs + tok[u] * xst[0] + h * xst[1], sl, on);
            rg[u].load(gs + tok[u] * gst[0] + h * gst[1], sl, on);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = base + u * G + gi, h = row - tok[u] * by.d;
            const bool pad = pos[u] < 0 || pos[u] >= a.d.max_pos;
            f32x2 x[4], y[4], gx[4], gy[4], sq = pk2(0.f, 0.f), dot = sq;
            if (u == 0 || tok[u] != tok[u > 0 ? u - 1 : 0])
                load_angles(a, sl, pos[u], c, s);
            if (pad) {   // no part in anything, whatever is there
                rx[u].clear();
                rg[u].clear();
            }
            rx[u].get(x, y);
            rg[u].get(gx, gy);
            if (sl.angle >= 0 && !pad)
                rotate<INTER, true>(gx, gy, c, s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sq = fma2(y[i], y[i], fma2(x[i], x[i], sq));
            const float ss = group_sum<LG>(sum2(sq));
            // (with eps 0 the r of a row of zeros would be infinite: its gradient is zero)
            const float r = ss == 0.f && a.d.eps == 0.f ? 0.f : rsqrtf(ss * g.inv_d + a.d.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // x becomes x r, g becomes g w
                x[i] = mul2(x[i], pk2(r, r));
                y[i] = mul2(y[i], pk2(r, r));
                ax[i] = fma2(gx[i], x[i], ax[i]);
                ay[i] = fma2(gy[i], y[i], ay[i]);
                gx[i] = mul2(gx[i], wx[i]);
                gy[i] = mul2(gy[i], wy[i]);
                dot = fma2(gy[i], y[i], fma2(gx[i], x[i], dot));
            }
            const float mean = -group_sum<LG>(sum2(dot)) * g.inv_d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                gx[i] = mul2(fma2(x[i], pk2(mean, mean), gx[i]), pk2(r, r));
                gy[i] = mul2(fma2(y[i], pk2(mean, mean), gy[i]), pk2(r, r));
            }
            if (row < n) {
                rg[u].set(gx, gy);
                rg[u].store(ds + tok[u] * dst[0] + h * dst[1], sl);
            }
        }
    }
    if (!part)
        return;
    // the groups of a warp, then the block's warps
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float vx = j & 1 ? hi2(ax[j / 2]) : lo2(ax[j / 2]), vy = j & 1 ? hi2(ay[j / 2]) : lo2(ay[j / 2]);
#pragma unroll
        for (int o = 16; o >= LG; o >>= 1) {
            vx += __shfl_xor_sync(0xffffffffu, vx, o);
            vy += __shfl_xor_sync(0xffffffffu, vy, o);
        }
        if (lane < LG) {
            if (sl.a >= 0)
                red[w][sl.a + j] = vx;
            if (sl.b >= 0)
                red[w][sl.b + j] = vy;
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i)
            v += red[i][d];
        part[(size_t)blockIdx.x * D + d] = v;
    }
}

// dq_weight, dk_weight: the blocks' parts added in a fixed order
__global__ void __launch_bounds__(1024) ssd_qk_weight_grad_kernel(const float *part, float *dqw, float *dkw, int D, int qblocks,
                                                                  int kblocks)
{
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx, key = blockIdx.y;
    const float *p = part + (key ? (size_t)qblocks * D : 0);
    const int n = key ? kblocks : qblocks;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float v = 0.f;
    if (col < D)
#pragma unroll 8
        for (int b = ty; b < n; b += 32)
            v += p[(size_t)b * D + col];
    red[ty][tx] = v;
    __syncthreads();
    float *out = key ? dkw : dqw;
    if (ty == 0 && col < D && out) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s += red[i][tx];
        out[col] = s;
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

template <typename K, typename... A>
cudaError_t launch(K *kernel, dim3 grid, int threads, cudaStream_t st, A... args)
{
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

// Blocks of either kind for `rows` rows per block; at most `most` in all, then
// shared out by rows.
RowGrid row_grid(const ssd_qk_dims_t &d, bool values, int rows, long long most)
{
    const long long q = (d.ntokens * d.nheads_q + rows - 1) / rows, k = (d.ntokens * d.nheads_k + rows - 1) / rows;
    const long long all = q + k * (values ? 2 : 1);
    RowGrid g{FastDiv(d.nheads_q), FastDiv(d.nheads_k), (int)q, (int)k, values ? (int)k : 0, 1.f / (float)d.headdim};
    if (all > most) {
        g.k = (int)std::max(most * k / all, 1ll);
        g.v = values ? g.k : 0;
        g.q = (int)std::max(most - g.k - g.v, 1ll);
    }
    return g;
}

RowGrid bwd_grid(const ssd_qk_dims_t &d)
{
    const int per = d.dtype == SSD_DTYPE_BF16 ? kRowsBwd<__nv_bfloat16> : kRowsBwd<float>;
    return row_grid(d, false, per * kThreads / lanes_for(d.headdim), (long long)kBwdPerSm * sm_count());
}

template <typename T, int LG>
cudaError_t fwd_lg(const QkArgs &a, cudaStream_t st)
{
    const RowGrid g = row_grid(a.d, a.kc != nullptr, kRowsFwd<T> * kThreads / LG, INT64_MAX);
    return launch(a.d.flags & SSD_ROPE_INTERLEAVED ? ssd_qk_norm_rope_kernel<T, LG, true> : ssd_qk_norm_rope_kernel<T, LG, false>,
                  dim3(g.q + g.k + g.v), kThreads, st, a, g);
}

template <typename T, int LG>
cudaError_t bwd_lg(const QkArgs &a, float *part, const RowGrid &g, cudaStream_t st)
{
    return launch(a.d.flags & SSD_ROPE_INTERLEAVED ? ssd_qk_norm_rope_bwd_kernel<T, LG, true> : ssd_qk_norm_rope_bwd_kernel<T, LG, false>,
                  dim3(g.q + g.k), kThreads, st, a, g, part);
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
cudaError_t bwd_t(const QkArgs &a, float *part, const RowGrid &g, cudaStream_t st)
{
    switch (lanes_for(a.d.headdim)) {
    case 1: return bwd_lg<T, 1>(a, part, g, st);
    case 2: return bwd_lg<T, 2>(a, part, g, st);
    case 4: return bwd_lg<T, 4>(a, part, g, st);
    case 8: return bwd_lg<T, 8>(a, part, g, st);
    default: return bwd_lg<T, 16>(a, part, g, st);
    }
}

}  // namespace

cudaError_t qk_fwd_launch(const QkArgs &a, cudaStream_t stream)
{
    SSD_NVTX_RANGE("qk_fwd_launch");
    // With eps 0 the 1 / rms of a row of zeros would be infinite.  The smallest numbers
    // keep it finite, so that the row stays zero, and are lost beside any normal mean
    // square (a comparison per row instead: 138.6 us for 137.4 on 32768 tokens).
    QkArgs b = a;
    b.d.eps = std::max(a.d.eps, 1e-44f);
    return a.d.dtype == SSD_DTYPE_BF16 ? fwd_t<__nv_bfloat16>(b, stream) : fwd_t<float>(b, stream);
}

size_t qk_bwd_workspace_bytes(const ssd_qk_dims_t &d)
{
    if (d.ntokens <= 0)
        return 0;
    const RowGrid g = bwd_grid(d);
    return (size_t)(g.q + g.k) * d.headdim * sizeof(float);
}

cudaError_t qk_bwd_launch(const QkArgs &a, void *workspace, cudaStream_t stream)
{
    SSD_NVTX_RANGE("qk_bwd_launch");
    float *part = static_cast<float *>(workspace);
    const RowGrid g = bwd_grid(a.d);
    cudaError_t e = a.d.dtype == SSD_DTYPE_BF16 ? bwd_t<__nv_bfloat16>(a, part, g, stream) : bwd_t<float>(a, part, g, stream);
    if (e == cudaSuccess && part)
        e = launch(ssd_qk_weight_grad_kernel, dim3((a.d.headdim + 31) / 32, 2), 1024, stream, (const float *)part, a.dqw, a.dkw,
                   (int)a.d.headdim, g.q, g.k);
    return e;
}

}  // namespace ssd
