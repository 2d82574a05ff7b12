// ssd_paged_attn_bf16_any.cu -- paged attention: bf16, any page and head size.
#include "ssd_paged_attn.cuh"

namespace ssd {

cudaError_t attn_launch_bf16_any(AttnParams &p, int mr, void *ws, cudaStream_t st)
{
    if (p.a.d.headdim <= 128)
        return mr == 32 ? launch_shares<Mma<2, 128, false, 1>, 4, 4, 2, true>(p, ws, st)
                        : launch_shares<Mma<1, 128, false, 1>, 4, 5, 2, true>(p, ws, st);
    return launch_shares<Mma<1, 256, false, 1>, 4, 5, 1, true>(p, ws, st);
}

cudaError_t attn_bf16_any_error(uint32_t *code) { return take_error(code); }

}  // namespace ssd
