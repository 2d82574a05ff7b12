// ssd_paged_attn.cu -- attention of new tokens over a paged key-value cache.
//
// One block per query row and head: its warps take the visible tokens in turn
// with a running maximum and sum each, and are joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float &o, float v) { o = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &o, float v) { o = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) ssd_paged_attn_simple_kernel(const __grid_constant__ AttnArgs a)
{
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, D = a.d.headdim;
    const long long row = blockIdx.x;
    const int h = blockIdx.y, kvh = h / (a.d.nheads / a.d.nkv);
    long long req = row;
    int pos = a.positions[row];
    if (a.start) {   // the last request that starts at or before the row
        int lo = -1, hi = (int)a.d.nreq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.start[mid] <= row)
                lo = mid;
            else
                hi = mid;
        }
        req = lo;
        if (lo < 0 || row >= a.start[a.d.nreq])
            pos = -1;
    }
    const int limit = a.d.max_pages * a.d.page_size;
    const int end = pos < 0 ? 0 : min(pos, limit - 1) + 1;
    const int first = a.d.window > 0 ? max(0, pos - a.d.window + 1) : 0;
    const T *q = static_cast<const T *>(a.q) + row * a.d.q_stride[0] + (long long)h * a.d.q_stride[1];
    float qv[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = lane + 32 * i;
        qv[i] = d < D ? to_f32(q[d]) : 0.f;
        o[i] = 0.f;
    }
    for (int t = first + w; t < end; t += kWarps) {
        const int p = t / a.d.page_size, off = t - p * a.d.page_size;
        const long long page = a.table[req * a.d.table_stride + p];
        if (page < 0 || page >= a.d.npages)
            continue;
        const T *k = static_cast<const T *>(a.kc) + page * a.d.kc_stride[0] + off * a.d.kc_stride[1] + kvh * a.d.kc_stride[2];
        const T *v = static_cast<const T *>(a.vc) + page * a.d.vc_stride[0] + off * a.d.vc_stride[1] + kvh * a.d.vc_stride[2];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d < D)
                s += qv[i] * to_f32(k[d]);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.d.scale;
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float keep = expf(m - base), e = expf(s - base);
        l = l * keep + e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d < D)
                o[i] = o[i] * keep + e * to_f32(v[d]);
        }
        m = mn;
    }
    if (lane == 0) {
        sm[w] = m;
        sl[w] = l;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        so[w][lane + 32 * i] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int i = 0; i < kWarps; ++i)
        mm = fmaxf(mm, sm[i]);
    const float base = mm == -INFINITY ? 0.f : mm;
    for (int i = 0; i < kWarps; ++i)
        ll += sl[i] * expf(sm[i] - base);
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    T *out = static_cast<T *>(a.out) + row * a.d.o_stride[0] + (long long)h * a.d.o_stride[1];
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float v = 0.f;
        for (int i = 0; i < kWarps; ++i)
            v += so[i][d] * expf(sm[i] - base);
        from_f32(out[d], v * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row * a.d.nheads + h] = ll == 0.f ? -INFINITY : base + logf(ll);
}

}  // namespace

size_t attn_workspace_bytes(const ssd_attn_dims_t &) { return 0; }

cudaError_t attn_launch(const AttnArgs &a, void *, cudaStream_t stream)
{
    SSD_NVTX_RANGE("attn_launch");
    const dim3 grid((unsigned)a.d.nrows, (unsigned)a.d.nheads);
    if (a.d.dtype == SSD_DTYPE_BF16)
        ssd_paged_attn_simple_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a);
    else
        ssd_paged_attn_simple_kernel<float><<<grid, kWarps * 32, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
