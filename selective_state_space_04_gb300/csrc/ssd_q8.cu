// ssd_q8.cu -- products of 8-bit integers with a scale per token and per output
// channel: y[t, n] = (sum_k a[t, k] w[n, k]) a_scale[t] w_scale[n], the sum exact in
// 32-bit integers.
//
// Weights are packed as the header says: tiles of 128 channels, in each the 16 bytes
// of 16 inner elements of all 128 channels side by side, so that a warp's loads are
// whole lines whatever K is.
#include <cuda_runtime.h>

#include <algorithm>

#include "ssd_internal.h"
#include "ssd_q8.h"

namespace ssd {
namespace {

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

namespace {

// Up to here the weights go through registers and mma.sync (8 tokens of 10576 x 2560: 8.4 us, with ssd_q8_mid.cu
// 12.1; 16 tokens 15.9, when they went through registers too, and 12.1).  Measured on these weights: of
// 16384 x 8192 8 tokens take 32.5 us here and 16 take 27.6 there, of 2560 x 5120 9.0 and 8.7.
constexpr long long kFew = 8;
// From here on both operands are widened first (256, 384 and 512 tokens of 10576 x 2560: 30.2, 37.5 and 53 us
// without; 288, 384 and 512 tokens 36.3, 37.0 and 39 to 43 us with).  Measured on these weights; what the widening
// costs goes by N K: 256 tokens of 16384 x 8192 take 77.6 us without and 288 take 133 with, of 2560 x 5120 17.8 and 26.9.
constexpr long long kMany = 257;

Q8Params params(const Q8Args &a)
{
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
    p.vec = ((uintptr_t)p.a & 7) == 0 && (p.sa % 8 == 0 || p.M == 1);
    p.yvec = ((uintptr_t)p.y & 15) == 0 && p.sy * (a.d.out_dtype == SSD_DTYPE_BF16 ? 2 : 4) % 16 == 0;
    return p;
}

}  // namespace

size_t q8_workspace_bytes(const ssd_q8_dims_t &d)
{
    const Q8Params p = params(Q8Args{nullptr, nullptr, nullptr, nullptr, nullptr, d});
    return d.M >= kMany ? q8_many_workspace_bytes(p) : d.M > kFew ? q8_mid_workspace_bytes(p) : 0;
}

cudaError_t q8_launch(const Q8Args &a, void *workspace, cudaStream_t st)
{
    SSD_NVTX_RANGE("q8_launch");
    const Q8Params p = params(a);
    const bool f32 = a.d.out_dtype == SSD_DTYPE_F32;
    if (p.M <= kFew)
        return q8_few_launch(p, f32, st);
    return p.M >= kMany ? q8_many_launch(p, f32, workspace, st) : q8_mid_launch(p, f32, workspace, st);
}

ssd_status_t q8_read_device_error(uint32_t *code)
{
    uint32_t many = 0;
    ssd_status_t s = q8_mid_read_device_error(code);
    if (s == SSD_OK)
        s = q8_many_read_device_error(&many);
    if (*code == 0)
        *code = many;
    return s;
}

}  // namespace ssd
