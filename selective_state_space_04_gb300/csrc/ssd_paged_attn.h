// ssd_paged_attn.h -- what the host side of the paged attention and its kernel
// translation units share.
#pragma once

#include <algorithm>
#include <cstdint>

#include "ssd_internal.h"

namespace ssd {

// exact floor(n / d) for 0 <= n < 2^31: (n * mul) >> sh
struct FastDiv {
    uint32_t mul, sh;
};

struct AttnParams {
    AttnArgs a;
    FastDiv page;
    float *part_o;      // [shares][2][MR][D] partial rows
    float *part_ml;     // [shares][2][MR][2] their maxima (of the scores before `f`) and sums
    int4 *desc;         // the cut tiles: first row, tokens | item << 8, first share, parts; x -1: none.  Shares of
                        // warps: [shares], of the tile that starts in a share; shares of CTAs: [most tiles x items]
    int ndesc;          // entries of it
    int of_head;        // shares of a key-value head (and head block)
    int nshares;        // of_head * items
    int few;            // at most kFewTiles tiles and requests, whose units fit 32 bits
    FastDiv by_items, by_tok;
    int group;          // query heads per key-value head
    int gh;             // query heads of a tile (group, or a part of it when it is larger than MR)
    int nhb;            // head blocks per key-value head
    int tok;            // most new tokens of a tile
    int most;           // tiles that the sizes allow at most
    int items;          // nkv * nhb: tiles of the same rows
    int seg;            // 16-byte segments per row of K or V
    uint32_t kpage, ktok, vpage, vtok;   // strides in 16 bytes
    long long khead, vhead;              // in bytes
    float f;            // |scale| log2(e), or 1 for scale 0
    int sign;           // of scale
    int sms;            // the device's SMs
};

constexpr int kFewTiles = 128;

inline FastDiv fast_div(int d)
{
    FastDiv f{0, 31};
    while ((1u << (f.sh - 31)) < (uint32_t)d)
        ++f.sh;
    f.mul = (uint32_t)((1ull << f.sh) / (uint32_t)d + 1);
    return f;
}

// tiles that the sizes allow at most (one per row, or per `tok` rows of a request)
inline long long most_tiles(const AttnParams &p)
{
    if (!p.a.start)
        return p.a.d.nrows;
    return std::max<long long>(1, std::min<long long>(p.a.d.nrows, p.a.d.nrows / p.tok + p.a.d.nreq));
}

// Shares of warps for at least two tiles (times key-value heads) per SM: below
// that a tile would be cut into more than four parts of warps, the join of
// which costs more than the CTAs' own joins.  Measured with shares of warps, of
// CTAs (8 key heads of 128, bf16): 128 tiles of 100..8000 tokens 55, 51 us; 256:
// 92.5, 91.5; 384: 131.4, 132.7; 400 tiles of 10..500: 19.7, 26.0.
inline bool solo_shares(const AttnParams &p) { return most_tiles(p) * p.items >= 2 * p.sms; }

constexpr int kWarps = 4;        // per CTA
constexpr int kMaxPerSm = 4;     // CTAs
constexpr int kMaxCtas = 1024;   // the workspace is sized for at most this many

// One launch of the main kernel and one of the join, for the variant whose tiles
// have `mr` rows.  bf16 with pages of whole 16 tokens and heads of 64, 128 or
// 256 elements; other bf16; fp32.
cudaError_t attn_launch_bf16(AttnParams &p, int mr, void *workspace, cudaStream_t stream);
cudaError_t attn_launch_bf16_any(AttnParams &p, int mr, void *workspace, cudaStream_t stream);
cudaError_t attn_launch_f32(AttnParams &p, int mr, void *workspace, cudaStream_t stream);

}  // namespace ssd
