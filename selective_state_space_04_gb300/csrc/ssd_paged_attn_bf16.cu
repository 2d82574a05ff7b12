// ssd_paged_attn_bf16.cu -- paged attention: bf16, pages of whole 16 tokens, heads
// of 64, 128 or 256 elements.
#include "ssd_paged_attn.cuh"

namespace ssd {

cudaError_t attn_launch_bf16(AttnParams &p, int mr, void *ws, cudaStream_t st)
{
    const int D = p.a.d.headdim;
    if (D == 64)
        return mr == 32 ? launch_shares<Mma<2, 64, true, 1>, 8, 8, 2, true>(p, ws, st)
                        : launch_shares<Mma<1, 64, true, 2>, 3, 3, 3, true>(p, ws, st);
    if (D == 128)
        return mr == 32 ? launch_shares<Mma<2, 128, true, 1>, 4, 4, 2, true>(p, ws, st)
                        : launch_shares<Mma<1, 128, true, 2>, 2, 2, 2, true>(p, ws, st);
    return launch_shares<Mma<1, 256, true, 1>, 4, 5, 1, true>(p, ws, st);
}

}  // namespace ssd
