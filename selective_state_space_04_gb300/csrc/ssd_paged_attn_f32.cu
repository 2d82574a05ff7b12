// ssd_paged_attn_f32.cu -- paged attention: fp32.  Bound by the cache's bytes up to
// 4 rows (32 requests of 100..8000 tokens, 8 key heads of 128, 1.06 GB: 171 us for one
// row or four, 6.2 TB/s), by the products for 8 (193 us).
#include "ssd_paged_attn.cuh"

namespace ssd {
namespace {

template <int MR>
cudaError_t launch_rows(AttnParams &p, void *ws, cudaStream_t st)
{
    const int D = p.a.d.headdim;
    if (D <= 64)
        return launch_shares<Simt<MR, 64, false>, 2, 2, 2, false>(p, ws, st);
    if (D <= 128)
        return launch_shares<Simt<MR, 128, false>, 2, 2, 2, false>(p, ws, st);
    return launch_shares<Simt<MR, 256, false>, MR == 8 ? 2 : 3, MR == 8 ? 2 : 3, 1, false>(p, ws, st);
}

}  // namespace

cudaError_t attn_launch_f32(AttnParams &p, int mr, void *ws, cudaStream_t st)
{
    switch (mr) {
    case 1: return launch_rows<1>(p, ws, st);
    case 2: return launch_rows<2>(p, ws, st);
    case 4: return launch_rows<4>(p, ws, st);
    default: return launch_rows<8>(p, ws, st);
    }
}

}  // namespace ssd
