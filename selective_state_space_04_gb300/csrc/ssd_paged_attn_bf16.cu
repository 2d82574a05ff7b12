// ssd_paged_attn_bf16.cu -- paged attention: bf16, pages of whole 16 tokens, heads
// of 64, 128 or 256 elements.
#include "ssd_paged_attn.cuh"

#ifndef V128_NT
#define V128_NT 2
#define V128_NU 2
#define V128_NUS 3
#define V128_MB 2
#endif
#ifndef V64_NT
#define V64_NT 2
#define V64_NU 3
#define V64_NUS 3
#define V64_MB 3
#endif

namespace ssd {

cudaError_t attn_launch_bf16(AttnParams &p, int mr, void *ws, cudaStream_t st)
{
    const int D = p.a.d.headdim;
    if (D == 64)
        return mr == 32 ? launch_shares<Mma<2, 64, true, 1>, 8, 8, 2, false>(p, ws, st)
                        : launch_shares<Mma<1, 64, true, V64_NT>, V64_NU, V64_NUS, V64_MB, false>(p, ws, st);
    if (D == 128)
        return mr == 32 ? launch_shares<Mma<2, 128, true, 1>, 4, 4, 2, false>(p, ws, st)
                        : launch_shares<Mma<1, 128, true, V128_NT>, V128_NU, V128_NUS, V128_MB, false>(p, ws, st);
    return launch_shares<Mma<1, 256, true, 1>, 4, 5, 1, false>(p, ws, st);
}

}  // namespace ssd
