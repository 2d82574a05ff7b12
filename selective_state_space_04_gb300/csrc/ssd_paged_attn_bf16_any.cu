// ssd_paged_attn_bf16_any.cu -- paged attention: bf16, any page and head size.
// Heads of 64 and 128 keep their compile-time size (64 requests of 100..8000
// tokens, pages of 24: heads of 64 99 us, of 128 175; heads of 80 146 us).
#include "ssd_paged_attn.cuh"

namespace ssd {

cudaError_t attn_launch_bf16_any(AttnParams &p, int mr, void *ws, cudaStream_t st)
{
    const int D = p.a.d.headdim;
    if (D == 64)
        return mr == 32 ? launch_shares<Mma<2, 64, true, 1>, 8, 8, 2, false>(p, ws, st)
                        : launch_shares<Mma<1, 64, true, 2>, 3, 3, 3, false>(p, ws, st);
    if (D == 128)
        return mr == 32 ? launch_shares<Mma<2, 128, true, 1>, 4, 4, 2, false>(p, ws, st)
                        : launch_shares<Mma<1, 128, true, 2>, 2, 2, 2, false>(p, ws, st);
    if (D < 128)
        return mr == 32 ? launch_shares<Mma<2, 128, false, 1>, 4, 4, 2, false>(p, ws, st)
                        : launch_shares<Mma<1, 128, false, 2>, 2, 2, 2, false>(p, ws, st);
    return launch_shares<Mma<1, 256, false, 1>, 4, 5, 1, false>(p, ws, st);
}

}  // namespace ssd
