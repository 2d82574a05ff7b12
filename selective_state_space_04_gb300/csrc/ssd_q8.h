// ssd_q8.h -- what the kernels of the 8-bit product share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssd_internal.h"

namespace ssd {

struct Q8Params {
    const int8_t *a, *w;          // [M, K] rows sa apart; packed
    const float *as, *ws;
    void *y;                      // [M, N] rows sy apart
    long long M, sa, sy;
    int N, K, k64, tiles;         // k64: slabs of 64 inner elements; tiles of 128 channels
    int vec;                      // a's rows are 8-byte aligned
    int yvec;                     // y's rows are 16-byte aligned
    // rows of a slab of the tokens' images
    __host__ __device__ long long padded() const { return (M + 127) / 128 * 128; }
};

// up to 8 tokens
cudaError_t q8_few_launch(const Q8Params &p, bool f32, cudaStream_t st);
// many tokens (workspace: 16-byte aligned)
size_t q8_many_workspace_bytes(const Q8Params &p);
cudaError_t q8_many_launch(const Q8Params &p, bool f32, void *workspace, cudaStream_t st);
// up to 256 tokens (workspace: 16-byte aligned)
size_t q8_mid_workspace_bytes(const Q8Params &p);
cudaError_t q8_mid_launch(const Q8Params &p, bool f32, void *workspace, cudaStream_t st);
// fp16 images of 128 rows x 64 elements, swizzled, from the first `wslabs` slabs of the weights (to
// wi, tile by tile) and all the tokens' (to ai, slab by slab, padded() rows each)
constexpr int kQ8Image = 128 * 128;   // bytes
cudaError_t q8_widen_launch(const Q8Params &p, uint8_t *wi, uint8_t *ai, long long wslabs, cudaStream_t st);
ssd_status_t q8_many_read_device_error(uint32_t *code);
ssd_status_t q8_mid_read_device_error(uint32_t *code);

#ifdef __CUDACC__
// Offset of 16-byte piece c of row r in a tile of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

// 4 8-bit integers to fp16, exactly: b + 128 below the bits of 1024 (spacing 1 there)
// is 1024 + 128 + b; 1152 is taken off again.
__device__ __forceinline__ void widen4(uint32_t u, uint32_t *f)
{
    const uint32_t v = u ^ 0x80808080u, lo = __byte_perm(v, 0x64646464u, 0x4140), hi = __byte_perm(v, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), off), b = __hsub2(*reinterpret_cast<const __half2 *>(&hi), off);
    f[0] = *reinterpret_cast<const uint32_t *>(&a);
    f[1] = *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void widen16(const uint4 &u, uint32_t *f)
{
    widen4(u.x, f);
    widen4(u.y, f + 2);
    widen4(u.z, f + 4);
    widen4(u.w, f + 6);
}

// a[t, k .. k + 15], zeros beyond M and K.  (Not through the read-only path: the launch before may write the
// tokens while this one lives.)
__device__ __forceinline__ uint4 load16(const Q8Params &p, long long t, int k)
{
    if (t >= p.M || k >= p.K)
        return make_uint4(0u, 0u, 0u, 0u);
    const int8_t *src = p.a + t * p.sa + k;
    if (p.vec && k + 16 <= p.K) {
        const uint2 lo = reinterpret_cast<const uint2 *>(src)[0], hi = reinterpret_cast<const uint2 *>(src)[1];
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (k + e < p.K)
            v[e / 4] |= (uint32_t)(uint8_t)src[e] << (8 * (e % 4));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// a[t, k .. k + 7], likewise
__device__ __forceinline__ uint2 load8(const Q8Params &p, long long t, int k)
{
    if (t >= p.M || k >= p.K)
        return make_uint2(0u, 0u);
    const int8_t *src = p.a + t * p.sa + k;
    if (p.vec && k + 8 <= p.K)
        return *reinterpret_cast<const uint2 *>(src);
    uint32_t v[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e < p.K)
            v[e / 4] |= (uint32_t)(uint8_t)src[e] << (8 * (e % 4));
    return make_uint2(v[0], v[1]);
}
#endif

}  // namespace ssd
