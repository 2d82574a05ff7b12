// ssd_paged_attn.cu -- paged attention: sizes, variants and parameters.  The
// kernels are in ssd_paged_attn.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ssd_paged_attn.h"

namespace ssd {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// How many query rows of a key-value head one request brings, as far as the
// sizes tell: the variant's rows per tile follow it.
long long rows_wanted(const ssd_attn_dims_t &d)
{
    const long long group = d.nheads / d.nkv;
    const long long tok = d.nreq > 0 ? (d.nrows + d.nreq - 1) / d.nreq : 1;
    return group * std::max<long long>(tok, 1);
}

// bf16: 32 rows where there are more than 16, so that the cache is read once for
// them (64 requests of 100..8000 tokens, 5 new ones each, groups of 4: 197 us; in
// tiles of 16 rows 319; groups of 16: 265 and 383.  Groups of 32 with one new token
// have few tiles and gain nothing: 49 either way).  Heads above 128 leave registers for 16 only.
// fp32: no more rows than there are, each costs its share of the products (one row:
// 172 us; as one of eight: 211).
int tile_rows(const ssd_attn_dims_t &d)
{
    const long long want = rows_wanted(d);
    if (d.dtype == SSD_DTYPE_BF16)
        return want > 16 && d.headdim <= 128 ? 32 : 16;
    return want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
}

}  // namespace

size_t attn_workspace_bytes(const ssd_attn_dims_t &d)
{
    const int grid = std::min(kMaxCtas, sm_count() * kMaxPerSm);
    // shares: as many as warps, or one per key-value head (and head block) where those are more
    const long long group = d.nheads / d.nkv, mr = tile_rows(d), items = d.nkv * ((group + mr - 1) / mr);
    const size_t shares = (size_t)std::max<long long>((long long)grid * kWarps, items);
    return shares * (2 * tile_rows(d) * (d.headdim + 2) * sizeof(float) + sizeof(int4));
}

cudaError_t attn_launch(const AttnArgs &a, void *workspace, cudaStream_t stream)
{
    SSD_NVTX_RANGE("attn_launch");
    AttnParams p{};
    p.a = a;
    const int mr = tile_rows(a.d), D = a.d.headdim, es = a.d.dtype == SSD_DTYPE_BF16 ? 2 : 4;
    p.group = a.d.nheads / a.d.nkv;
    p.nhb = (p.group + mr - 1) / mr;
    p.gh = (p.group + p.nhb - 1) / p.nhb;
    p.tok = a.start ? std::max(1, mr / p.gh) : 1;
    p.items = a.d.nkv * p.nhb;
    p.seg = D * es / 16;
    // (a stride that no second page, token or head uses may be anything)
    auto used = [](int64_t n, int64_t stride) { return n > 1 ? stride : 0; };
    p.kpage = (uint32_t)(used(a.d.npages, a.d.kc_stride[0]) * es / 16);
    p.vpage = (uint32_t)(used(a.d.npages, a.d.vc_stride[0]) * es / 16);
    p.ktok = (uint32_t)(used(a.d.page_size, a.d.kc_stride[1]) * es / 16);
    p.vtok = (uint32_t)(used(a.d.page_size, a.d.vc_stride[1]) * es / 16);
    p.khead = used(a.d.nkv, a.d.kc_stride[2]) * es;
    p.vhead = used(a.d.nkv, a.d.vc_stride[2]) * es;
    // scores are kept as q.k times the scale's sign, so that their maximum is that of the scaled ones
    p.sign = a.d.scale > 0.f ? 1 : a.d.scale < 0.f ? -1 : 0;
    p.f = p.sign ? fabsf(a.d.scale) * kLog2e : 1.f;
    p.page = fast_div(a.d.page_size);
    p.by_items = fast_div(p.items);
    p.by_tok = fast_div(p.tok);
    p.most = (int)most_tiles(p);
    p.few = most_tiles(p) <= kFewTiles && a.d.nreq <= kFewTiles &&
            kFewTiles * ((int64_t)a.d.page_size * a.d.max_pages / 16 + 8) < (INT64_C(1) << 31);
    p.sms = sm_count();
    if (a.d.dtype == SSD_DTYPE_F32)
        return attn_launch_f32(p, mr, workspace, stream);
    const bool sized = a.d.page_size % 16 == 0 && (D == 64 || D == 128 || D == 256);
    return sized ? attn_launch_bf16(p, mr, workspace, stream) : attn_launch_bf16_any(p, mr, workspace, stream);
}

}  // namespace ssd
