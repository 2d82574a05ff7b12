// ssd_paged_attn_bf16_any.cu -- paged attention: bf16, any page and head size.
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
