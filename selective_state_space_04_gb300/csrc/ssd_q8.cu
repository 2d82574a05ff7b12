// ssd_q8.cu -- products of 8-bit integers with a scale per token and per output
// channel: y[t, n] = (sum_k a[t, k] w[n, k]) a_scale[t] w_scale[n], the sum exact in
// 32-bit integers.
//
// Weights are packed as the header says: tiles of 128 channels, in each the 16 bytes
// of 16 inner elements of all 128 channels side by side, so that a warp's loads are
// whole lines whatever K is.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kTokens = 8;   // tokens of a block

struct Q8Params {
    const int8_t *a, *w;
    const float *as, *ws;
    void *y;
    long long M, sa, sy, items;
    int N, K, k64, tiles;
};

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// One block: 128 channels (a thread each) of kTokens tokens.
template <typename T>
__global__ void __launch_bounds__(128) ssd_q8_kernel(Q8Params p)
{
    __shared__ __align__(16) int8_t s[kTokens][64];
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        const int tile = (int)(item % p.tiles), n = tile * 128 + threadIdx.x;
        const long long t0 = item / p.tiles * kTokens;
        int acc[kTokens] = {};
        for (int kb = 0; kb < p.k64; ++kb) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTokens * 64; i += 128) {
                const long long t = t0 + i / 64;
                const int k = kb * 64 + i % 64;
                s[i / 64][i % 64] = t < p.M && k < p.K ? p.a[t * p.sa + k] : (int8_t)0;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 w = *reinterpret_cast<const uint4 *>(p.w + (((size_t)tile * p.k64 + kb) * 4 + c) * 2048 + threadIdx.x * 16);
#pragma unroll
                for (int t = 0; t < kTokens; ++t) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(&s[t][c * 16]);
                    acc[t] = __dp4a((int)w.x, (int)a.x, acc[t]);
                    acc[t] = __dp4a((int)w.y, (int)a.y, acc[t]);
                    acc[t] = __dp4a((int)w.z, (int)a.z, acc[t]);
                    acc[t] = __dp4a((int)w.w, (int)a.w, acc[t]);
                }
            }
        }
        if (n < p.N)
            for (int t = 0; t < kTokens && t0 + t < p.M; ++t)
                static_cast<T *>(p.y)[(t0 + t) * p.sy + n] = from_f32<T>((float)acc[t] * p.as[t0 + t] * p.ws[n]);
    }
}

// packed[tile][k / 16][channel][k % 16]: one thread per 16 bytes
__global__ void __launch_bounds__(256) ssd_q8_pack_kernel(const int8_t *w, int8_t *packed, int N, int K, long long stride,
                                                          long long chunks)
{
    const int k16s = (K + 63) / 64 * 4;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long long)gridDim.x * 256) {
        const long long rest = i / 128, n = rest / k16s * 128 + i % 128;
        const int k0 = (int)(rest % k16s) * 16;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (n < N)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k0 + e < K)
                    v[e / 4] |= (uint32_t)(uint8_t)w[n * stride + k0 + e] << (8 * (e % 4));
        reinterpret_cast<uint4 *>(packed)[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

}  // namespace

cudaError_t q8_pack_launch(const int8_t *w, int8_t *packed, const ssd_q8_dims_t &d, cudaStream_t st)
{
    SSD_NVTX_RANGE("q8_pack_launch");
    const long long chunks = SSD_Q8_PACKED_BYTES(d.N, d.K) / 16;
    ssd_q8_pack_kernel<<<(unsigned)std::min<long long>((chunks + 255) / 256, 65536), 256, 0, st>>>(w, packed, d.N, d.K, d.a_stride, chunks);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

size_t q8_workspace_bytes(const ssd_q8_dims_t &) { return 0; }

cudaError_t q8_launch(const Q8Args &a, void *, cudaStream_t st)
{
    SSD_NVTX_RANGE("q8_launch");
    if (a.d.M == 0)
        return cudaSuccess;
    Q8Params p;
    p.a = a.a;
    p.w = a.packed;
    p.as = a.a_scale;
    p.ws = a.w_scale;
    p.y = a.y;
    p.M = a.d.M;
    p.sa = a.d.a_stride;
    p.sy = a.d.y_stride;
    p.N = a.d.N;
    p.K = a.d.K;
    p.k64 = (p.K + 63) / 64;
    p.tiles = (p.N + 127) / 128;
    p.items = (p.M + kTokens - 1) / kTokens * p.tiles;
    const unsigned grid = (unsigned)std::min<long long>(p.items, 1 << 20);
    if (a.d.out_dtype == SSD_DTYPE_F32)
        ssd_q8_kernel<float><<<grid, 128, 0, st>>>(p);
    else
        ssd_q8_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
