// ssd_paged_attn.cuh -- attention of new tokens over a paged key-value cache.
//
// A tile is up to MR query rows that read the same keys: the query heads of one
// key-value head for one or several consecutive new tokens of a request.  The
// tile's visible positions are cut into units of 16 or 32 tokens.  The units of
// all tiles, laid end to end, are dealt out in equal contiguous shares, whatever
// the requests' lengths, the same shares for every key-value head.  Neighbouring
// warps (or CTAs) take the same share of neighbouring heads, so that a token's
// heads, which lie side by side in a token-major cache, are read at about the
// same time.  The CTAs that fit the GPU at once stay for the whole launch.  A warp
// streams its units through a ring of shared-memory slots of its own, K and V
// halves in turn, and keeps a running maximum, sum and output rows in registers:
// no barrier stands between loads and arithmetic, and loads run ahead across tile
// boundaries.
//
// Shares belong to warps, or to CTAs, whose warps then take units in turn and
// are joined in shared memory at the end of a tile (many tiles, or few: see
// solo_shares).  A tile that lies in one share is finished there; one that is cut
// leaves partial results (maximum, sum, unnormalised rows), which a second
// launch joins in the order of their shares.
//
// What bounds it.  Up to 16 rows per tile: the cache's bytes, each read once
// (bf16 heads of 128, 8 of them, 128 requests of 1..4096 tokens, 1.08 GB: 173 us,
// 6.2 TB/s; 128 requests of 500..12000 with 4 new tokens each: 505 us, 6.5 TB/s).
// Little work: a chain of dependent steps -- finding the share, table entry, keys,
// values, join -- of 7 to 10 us (one request of 1000 tokens: 8 us).  More rows:
// the products and the softmax beside them, on two warps per scheduler, which is
// what the output rows' registers leave (64 requests of 100..8000, 20 rows: 195 us,
// 5.5 TB/s; a whole prompt of 8192 tokens, 32 heads of 128: 2.73 ms, 0.20 PFLOP/s).
//
// The running form: with s = q.k (its sign that of the scaled score), f =
// |scale| log2(e), m = max s so far, p = 2^(f (s - m)), l = sum p, o = sum p v;
// when m grows by d, l and o are scaled by 2^(-f d).  out = o / l, lse =
// ln 2 (f m + log2 l).  Everywhere the difference is taken first and then scaled:
// equal maxima give a factor of exactly 1, and however large the scores are, no
// weight is off by more than the scores themselves (a difference of two scaled
// scores would carry the rounding of each, 2^-24 of their size, into the
// exponent).  The addition that a fused f s - f m would save costs nothing that
// shows (a prompt of 8192 tokens 2749 us, fused 2762; fp32, 8 rows, 191 and 191).
//
// bf16: both products run on mma.sync m16n8k16 (scores: 16 query rows x 8
// tokens; output: 16 rows x 8 elements over 16 tokens).  A score tile's
// accumulator registers are, as they stand, the second product's A operand.
// The weights p enter it as two bf16 terms, so that they carry 16 bits: one
// bf16 term would add an error as large as the output's own rounding, and saves
// little (32 requests of 100..8000 tokens, 32 rows: 2 of 52 us).
// fp32: fp32 FMA (see Simt below).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "ssd_paged_attn.h"

namespace ssd {
namespace {

constexpr int kThreads = 32 * kWarps;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kSlack = 8.f;   // in powers of 2

__device__ __forceinline__ int div_fast(const FastDiv &f, int n) { return (int)(((uint64_t)(uint32_t)n * f.mul) >> f.sh); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes, or zeros when !on (nothing is read then, but the address must be valid all the same)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- the walk over tiles, items and units ---------------------------------

// One tile of query rows: nq tokens from row `row` of request `req`; the tokens
// they see lie in [first, end), in `units` units from unit `ub` on.
struct Tile {
    int req, j, row, nq, rows_left;   // j: tile of the request; rows_left: the request's rows after this tile
    int first, end, ub, units;
};

// Positions are any int32, and the last one seen may be 2^31 - 2: neither may
// overflow.  The end of what the row at `pos` sees, and its first position:
__device__ __forceinline__ int seen_end(const AttnParams &p, int pos)
{
    return pos < 0 ? 0 : min(pos, p.a.d.max_pages * p.a.d.page_size - 1) + 1;
}
__device__ __forceinline__ int seen_first(const AttnParams &p, int pos)
{
    return p.a.d.window > 0 && pos >= p.a.d.window ? pos - p.a.d.window + 1 : 0;
}

// the extent from the positions of the first and the last row
template <int UT>
__device__ __forceinline__ void tile_extent(const AttnParams &p, Tile &t, int p0, int p1)
{
    t.end = seen_end(p, p1);
    t.first = min(seen_first(p, p0), t.end);
    t.ub = t.first / UT;
    const int units = (int)(((uint32_t)t.end + UT - 1) / UT);
    t.units = max(1, units - t.ub);   // (a tile that sees nothing still writes its rows)
}

// rows [s, e) of request r, clamped to the rows there are
__device__ __forceinline__ void request_rows(const AttnParams &p, int r, int &s, int &e)
{
    const int n = (int)p.a.d.nrows;
    s = min(max(p.a.start[r], 0), n);
    e = min(max(p.a.start[r + 1], s), n);
}

template <int UT>
__device__ __forceinline__ void set_tile(const AttnParams &p, Tile &t, int req, int j)
{
    t.req = req;
    t.j = j;
    if (p.a.start) {
        int s, e;
        request_rows(p, req, s, e);
        t.row = s + j * p.tok;
        t.nq = min(p.tok, e - t.row);
        t.rows_left = e - t.row - t.nq;
    } else {
        t.row = req;
        t.nq = 1;
        t.rows_left = 0;
    }
    const int p0 = p.a.positions[t.row];
    tile_extent<UT>(p, t, p0, t.nq > 1 ? p.a.positions[t.row + t.nq - 1] : p0);
}

// the next tile (there is one)
template <int UT>
__device__ __forceinline__ void next_tile(const AttnParams &p, Tile &t)
{
    if (t.rows_left > 0) {
        set_tile<UT>(p, t, t.req, t.j + 1);
        return;
    }
    int r = t.req + 1;
    if (p.a.start) {
        int s, e;
        while (r < (int)p.a.d.nreq - 1) {
            request_rows(p, r, s, e);
            if (e > s)
                break;
            ++r;
        }
    }
    set_tile<UT>(p, t, r, 0);
}

// A place in a share: a tile and the number of its first unit.
struct Cursor {
    Tile t;
    int tile;   // counted over all requests
    long long lin;
};

template <int UT>
__device__ __forceinline__ void advance(const AttnParams &p, Cursor &c)
{
    c.lin += c.t.units;
    ++c.tile;
    next_tile<UT>(p, c.t);
}

// a / b for a >= 0, b > 0: in 32 bits where they fit (a 64-bit division takes some
// hundred cycles)
__device__ __forceinline__ long long div_units(long long a, long long b)
{
    return ((unsigned long long)a | (unsigned long long)b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// ---- block scan for the schedule ------------------------------------------

__device__ __forceinline__ long long block_exclusive(long long v, long long *total, long long *tmp)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += u;
    }
    __syncthreads();
    if (lane == 31)
        tmp[w] = inc;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < w)
            before += tmp[i];
        all += tmp[i];
    }
    *total = all;
    return before + inc - v;
}

struct Found {
    int req, j, tile;
    long long lin;   // the linear unit where the tile's first item begins
};

struct Shares {
    long long total, per;   // units of a key-value head, and of a share
    long long ntiles;
    bool chunks;            // a share is at most `per` units of one tile, whose next one begins with the next share
};

// For at most kFewTiles tiles: each warp sums all tiles' units (four tiles a lane)
// and finds its own share's beginning, without a barrier (one request of 1000
// tokens: 7.9 us instead of 8.6 by way of `locate`).  `list` (shared memory
// of the warp, kFewTiles entries) is used when there is a start array.
template <int UT, bool SOLO>
__device__ __forceinline__ Shares locate_few(const AttnParams &p, int j, Cursor &cur, int4 *list)
{
    const int lane = threadIdx.x & 31;
    int n = (int)p.a.d.nrows;
    if (p.a.start) {   // first row, tokens, tile of the request and its rows left | request, of each tile
        int s[4], e[4], cnt[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = e[i] = 0;
            if (4 * lane + i < (int)p.a.d.nreq)
                request_rows(p, 4 * lane + i, s[i], e[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine += cnt[i] = div_fast(p.by_tok, e[i] - s[i] + p.tok - 1);
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o)
                at += u;
        }
        n = min(__shfl_sync(0xffffffffu, at, 31), kFewTiles);
        at -= mine;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            for (int k = 0; k < cnt[i] && at < kFewTiles; ++k, ++at) {
                const int row = s[i] + k * p.tok, nq = min(p.tok, e[i] - row);
                list[at] = make_int4(row, nq | (4 * lane + i) << 8, k, e[i] - row - nq);
            }
        __syncwarp();
    }
    int pos[4], last[4], units[4], sum = 0, padded = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pos[i] = last[i] = -1;
        const int tile = 4 * lane + i;
        if (tile < n) {
            const int4 d = p.a.start ? list[tile] : make_int4(tile, 1, 0, 0);
            pos[i] = last[i] = p.a.positions[d.x];
            if ((d.y & 0xff) > 1)
                last[i] = p.a.positions[d.x + (d.y & 0xff) - 1];
        }
    }
    Tile t{0, 0, 0, 1, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        tile_extent<UT>(p, t, pos[i], last[i]);
        units[i] = 4 * lane + i < n ? t.units : 0;
        sum += units[i];
        padded += (units[i] + kWarps - 1) / kWarps * kWarps;
    }
    int inc = sum, incp = padded = min(padded, 1 << 20);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o), v = SOLO ? 0 : __shfl_up_sync(0xffffffffu, incp, o);
        if (lane >= o) {
            inc += u;
            incp += v;
        }
    }
    int total = __shfl_sync(0xffffffffu, inc, 31);
    // So little work that each CTA can have at most a unit per warp, of one tile
    // (two tiles of a CTA would be one after the other): tiles begin with shares.
    // 17 requests of two units or three: 7.3 us; four units to a CTA, across tiles: 13.8.
    const int whole = SOLO ? 0 : __shfl_sync(0xffffffffu, incp, 31);
    const bool chunks = !SOLO && whole <= p.of_head * kWarps;
    if (chunks) {
        total = whole;
        sum = padded;
        inc = incp;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            units[i] = (units[i] + kWarps - 1) / kWarps * kWarps;
    }
    const int per = max(SOLO ? 1 : kWarps, (int)(((unsigned)total + p.of_head - 1) / (unsigned)p.of_head));
    const Shares sh{total, per, n, chunks};
    const int u0 = (int)min((long long)j * per, (long long)total);   // (total: the share is empty)
    // the last lane that begins at or before u0, and the row of its four
    const int from = 31 - __clz(__ballot_sync(0xffffffffu, inc - sum <= u0));
    int lin = inc - sum, tile = 4 * lane, p0 = pos[0], p1 = last[0];
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (tile == 4 * lane + i && units[i + 1] > 0 && u0 >= lin + units[i]) {
            lin += units[i];
            ++tile;
            p0 = pos[i + 1];
            p1 = last[i + 1];
        }
    t.req = t.row = cur.tile = __shfl_sync(0xffffffffu, tile, from);
    p0 = __shfl_sync(0xffffffffu, p0, from);
    p1 = __shfl_sync(0xffffffffu, p1, from);
    cur.lin = __shfl_sync(0xffffffffu, lin, from);
    if (p.a.start) {
        const int4 d = list[cur.tile];
        t.row = d.x;
        t.nq = d.y & 0xff;
        t.req = d.y >> 8;
        t.j = d.z;
        t.rows_left = d.w;
        __syncwarp();   // (the list's memory is the ring's)
    }
    tile_extent<UT>(p, t, p0, p1);
    cur.t = t;
    return sh;
}

// Finds where share j of a head begins (found[i] for warp i's share, or
// found[0]).  Every CTA sums all tiles' units (a contiguous run of tiles per
// thread); the thread whose run holds a share's first unit finds its tile.
// `counts` (shared memory, nreq + 1 ints) is used when there is a start array.
template <int UT, bool SOLO>
__device__ __forceinline__ Shares locate(const AttnParams &p, int *counts, long long *tmp, Found *found)
{
    const int tid = threadIdx.x, nreq = (int)p.a.d.nreq;
    long long ntiles = p.a.d.nrows;
    if (p.a.start) {
        const int run = (nreq + kThreads - 1) / kThreads, r0 = min(tid * run, nreq), r1 = min(r0 + run, nreq);
        long long n = 0, all;
        for (int r = r0; r < r1; ++r) {
            int s, e;
            request_rows(p, r, s, e);
            n += ((uint32_t)(e - s) + p.tok - 1) / p.tok;
        }
        long long at = block_exclusive(n, &all, tmp);
        for (int r = r0; r < r1; ++r) {
            int s, e;
            request_rows(p, r, s, e);
            counts[r] = (int)min(at, (long long)p.most);   // (a start array that descends could have more)
            at += ((uint32_t)(e - s) + p.tok - 1) / p.tok;
        }
        ntiles = min(all, (long long)p.most);
        if (tid == 0)
            counts[nreq] = (int)ntiles;
        __syncthreads();
    }
    const long long run = (ntiles + kThreads - 1) / kThreads, t0 = min((long long)tid * run, ntiles), t1 = min(t0 + run, ntiles);
    // the run's first tile
    Found f{0, 0, 0, 0};
    if (t0 < t1) {
        if (p.a.start) {
            int lo = 0, hi = nreq;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (counts[mid] <= t0)
                    lo = mid;
                else
                    hi = mid;
            }
            f.req = lo;
            f.j = (int)(t0 - counts[lo]);
        } else
            f.req = (int)t0;
    }
    long long n = 0;
    Tile t;
    for (long long i = t0; i < t1; ++i) {
        if (i == t0)
            set_tile<UT>(p, t, f.req, f.j);
        else
            next_tile<UT>(p, t);
        n += t.units;
    }
    long long sum;
    const long long before = block_exclusive(n, &sum, tmp);
    constexpr int kOwn = SOLO ? kWarps : 1;   // shares of a CTA at a time
    Shares sh;
    sh.total = sum;
    sh.ntiles = ntiles;
    sh.chunks = false;
    sh.per = max((long long)(SOLO ? 1 : kWarps), div_units(sum + p.of_head - 1, p.of_head));
    if (t0 < t1) {
        long long lin = before, tile = t0;
        const long long end = before + n;
        bool at_start = false;
        for (int i = 0; i < kOwn; ++i) {
            // (more heads than CTAs' shares: one share per head, from the first unit on)
            const int share = blockIdx.x * kOwn + i, j = p.of_head == 1 ? 0 : div_fast(p.by_items, share);
            const long long u0 = j * sh.per;
            if (u0 < before || u0 >= end)
                continue;
            if (!at_start) {   // (the walk goes on from share to share)
                set_tile<UT>(p, t, f.req, f.j);
                at_start = true;
            }
            while (u0 >= lin + t.units) {
                lin += t.units;
                next_tile<UT>(p, t);
                ++tile;
            }
            found[i].req = t.req;
            found[i].j = t.j;
            found[i].tile = (int)tile;
            found[i].lin = lin;
        }
    }
    __syncthreads();
    return sh;
}

// ---- the loader -------------------------------------------------------------

// How a unit gets into the ring, always by 16-byte copies, each lane at a fixed
// segment of every row.  ALIGNED: 16 aligned tokens never cross a page, so that one
// offset serves 16 rows; else each row's offset comes from the lane that looked its
// page up (in ALIGNED's place: 128 requests of 1..4096 tokens, heads of 128, 175 us
// instead of 172; one of 1000, 8.1 instead of 7.8; heads of 64 no difference).  One
// bulk copy per row was slower for bf16 (a row per some 9 cycles and SM: heads of
// 64, 64 requests of 100..8000, 184 us instead of 99) and fp32 heads of 64 (198
// requests of 1..3971: 345 instead of 267), though not for fp32 heads of 128 with
// one query head each (157 instead of 169).

// Streams a warp's units into its ring, K halves and V halves in turn.
template <typename T, int DP, bool EX, bool ALIGNED, int UT>
struct Loader {
    static constexpr int kSegMax = DP * (int)sizeof(T) / 16;
    static constexpr int kSub = ALIGNED ? UT / 16 : 1;
    // a lane's rows lie kRows apart
    static constexpr int kRows = 32 / kSegMax > 0 ? 32 / kSegMax : 1;    // rows per instruction
    static constexpr int kParts = kSegMax / 32 > 0 ? kSegMax / 32 : 1;   // instructions per row
    static constexpr int kStride = (kSegMax | 1) * 16;
    static constexpr uint32_t kAll = UT == 16 ? 0xffffu : 0xffffffffu;
    Cursor c;
    int u, u_end;          // the unit within the tile (-1: none left); the share's units of the tile
    long long u1;          // end of the share
    const char *kb, *vb;   // the key-value head in the caches (ALIGNED: at the lane's row and segment)
    const int32_t *table;  // the request's row
    int page;              // table entry read ahead (of the lane's 16 tokens, or of its token)
    uint32_t mask;         // the unit's tokens that are to be read
    // offsets in 16 bytes: of the first token of each 16, or of the lane's token
    uint64_t koff[kSub], voff[kSub];

    __device__ __forceinline__ void set_head(const AttnParams &p, int kvh, int lane)
    {
        kb = static_cast<const char *>(p.a.kc) + kvh * p.khead;
        vb = static_cast<const char *>(p.a.vc) + kvh * p.vhead;
        if (ALIGNED) {
            kb += (lane / kSegMax) * (long long)p.ktok * 16 + (lane % kSegMax) * 16;
            vb += (lane / kSegMax) * (long long)p.vtok * 16 + (lane % kSegMax) * 16;
        }
    }
    __device__ __forceinline__ void set_tile_end(const AttnParams &p)
    {
        u_end = (int)min((long long)c.t.units, u1 - c.lin);
        table = p.a.table + (long long)c.t.req * p.a.d.table_stride;
    }
    // the unit `by` further on in the share
    __device__ __forceinline__ void skip(const AttnParams &p, int by)
    {
        u += by;
        while (u >= u_end) {
            if (c.lin + u >= u1) {
                u = -1;
                return;
            }
            u -= c.t.units;
            advance<UT>(p, c);
            set_tile_end(p);
        }
    }
    __device__ __forceinline__ void fetch_page(const AttnParams &p, int lane)
    {
        page = -1;
        if (u >= 0) {
            const int tok = (c.t.ub + u) * UT + (ALIGNED ? (kSub > 1 ? lane & 16 : 0) : lane % UT);
            if (tok < c.t.end)   // (16 tokens are in the page of the first of them)
                page = table[div_fast(p.page, tok)];   // (not through the read-only path: the launch before may write it)
        }
    }
    __device__ __forceinline__ void offsets(const AttnParams &p, int lane)
    {
        const int tok0 = (c.t.ub + u) * UT, tok = tok0 + lane % UT;
        const bool there = (unsigned)page < (unsigned)p.a.d.npages;
        mask = __ballot_sync(0xffffffffu, tok >= c.t.first && tok < c.t.end && there);
        if (UT == 16)
            mask &= 0xffffu;
#pragma unroll
        for (int b = 0; b < kSub; ++b) {
            // (an entry out of range masks its tokens: nothing is read at its offset)
            const uint32_t pg = (uint32_t)max(kSub > 1 ? __shfl_sync(0xffffffffu, page, 16 * b) : page, 0);
            const int at = ALIGNED ? tok0 + 16 * b : tok;
            const uint32_t off = at - div_fast(p.page, at) * p.a.d.page_size;
            koff[b] = (uint64_t)pg * p.kpage + (uint64_t)off * p.ktok;
            voff[b] = (uint64_t)pg * p.vpage + (uint64_t)off * p.vtok;
        }
    }
    // one half (UT tokens of K or V) into a ring slot; rows that are not read become zero
    __device__ __forceinline__ void copy(const AttnParams &p, const char *base, const uint64_t (&off)[kSub], uint32_t tok16,
                                         uint32_t slot, int lane)
    {
        const uint32_t dst = slot + (lane / kSegMax) * kStride + (lane % kSegMax) * 16;
        const uint64_t step = (uint64_t)tok16 * (kRows * 16);
        if (mask == kAll) {
#pragma unroll
            for (int b = 0; b < kSub; ++b) {
                const char *s = base + (off[b] << 4);
#pragma unroll
                for (int i = 0; i < 16 / kRows; ++i, s += step)
#pragma unroll
                    for (int x = 0; x < kParts; ++x)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         dst + (16 * b + i * kRows) * kStride + x * 512), "l"(s + x * 512) : "memory");
            }
        } else {
            const uint32_t mine = mask >> (lane / kSegMax);
#pragma unroll
            for (int b = 0; b < kSub; ++b) {
                const char *s = base + (off[b] << 4);
#pragma unroll
                for (int i = 0; i < 16 / kRows; ++i, s += step) {
                    const bool on = (mine >> (16 * b + i * kRows)) & 1;
#pragma unroll
                    for (int x = 0; x < kParts; ++x)
                        cp_async16(dst + (16 * b + i * kRows) * kStride + x * 512,
                                   on ? s + x * 512 : static_cast<const char *>(p.a.q), on);
                }
            }
        }
    }
    // ... of any page, a row's offset taken from its lane; the lanes of segments past
    // the head's elements are idle
    __device__ __forceinline__ void copy_any(const AttnParams &p, const char *base, uint64_t off, uint32_t slot, int lane)
    {
        const int r0 = lane / kSegMax, c = lane % kSegMax;
        const uint32_t dst = slot + r0 * kStride + c * 16, mine = mask >> r0;
        const char *src[UT / kRows];
        // (sources first: the exchanges between lanes would stand between the copies)
#pragma unroll
        for (int i = 0; i < UT / kRows; ++i) {
            const uint64_t from = __shfl_sync(0xffffffffu, off, r0 + i * kRows);
            src[i] = base + (from << 4) + c * 16;
        }
#pragma unroll
        for (int x = 0; x < kParts; ++x)
            if (EX || c + 32 * x < p.seg) {
#pragma unroll
                for (int i = 0; i < UT / kRows; ++i) {
                    const bool on = (mine >> (i * kRows)) & 1;
                    cp_async16(dst + i * kRows * kStride + x * 512, on ? src[i] + x * 512 : static_cast<const char *>(p.a.q), on);
                }
            }
    }
};

// ---- the arithmetic: bf16 on mma.sync --------------------------------------

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// the two bf16, infinities and NaN as the largest finite value of their sign
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v)
{
    uint32_t r;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7f7f7f7fu));
    return r;
}

// the largest of the warps' maxima of row r (0 when no warp saw a token)
template <int MR>
__device__ __forceinline__ float joint_max(const float *ml, int r)
{
    float v = ml[2 * r];
#pragma unroll
    for (int i = 1; i < kWarps; ++i)
        v = fmaxf(v, ml[(i * MR + r) * 2]);
    return v == -INFINITY ? 0.f : v;
}

// NM: tiles of 16 query rows; DP: the head's elements, rounded up (EXACT: as
// they are); NT: 16-token halves of a unit.  A lane holds results of rows
// lane / 4 and lane / 4 + 8 of each tile.
template <int NM, int DP, bool EX, int NT>
struct Mma {
    using T = __nv_bfloat16;
    static constexpr int MR = 16 * NM, kDim = DP, kUnit = 16 * NT;
    static constexpr bool kExact = EX;
    // Query rows stay in registers, but for 16 KB of output rows per warp and
    // more (256 of a lane's registers are not enough for both): then in shared
    // memory, read anew for each unit.
    static constexpr bool kQSmem = NM * DP >= 256;
    static constexpr int kQStride = (DP / 8 | 1) * 16;
    static constexpr int kQBytes = kQSmem ? MR * kQStride : 0;   // per warp
    uint32_t q[kQSmem ? 1 : NM][kQSmem ? 1 : DP / 16][4];
    char *qs;
    float o[NM][DP / 8][4];
    float s[NM][2 * NT][4];
    float m[NM][2], l[NM][2];   // m: the running maximum of q.k (of -q.k for a negative scale)
    int lo[NM][2], hi[NM][2];   // positions a row sees

    __device__ __forceinline__ static int dim(const AttnParams &p) { return EX ? DP : p.a.d.headdim; }
    // of a ring slot: an odd number of segments, so that 8 rows' segments lie in different banks
    static constexpr int kRowBytes = (DP / 8 | 1) * 16;

    __device__ __forceinline__ void begin(const AttnParams &p, const Tile &t, int item, int lane)
    {
        const int kvh = p.nhb == 1 ? item : item / p.nhb, hb = item - kvh * p.nhb, D = dim(p);
        const int h0 = hb * p.gh, nh = min(p.gh, p.group - h0), rows = t.nq * nh;
        const uint32_t keep = p.sign == 0 ? 0u : 0xffffffffu, flip = p.sign < 0 ? 0x80008000u : 0u;
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = mt * 16 + x * 8 + (lane >> 2), rr = min(r, rows - 1), j = t.nq == 1 ? 0 : rr / nh, g = rr - j * nh;
                const int pos = p.a.positions[t.row + j];
                hi[mt][x] = seen_end(p, pos);
                lo[mt][x] = seen_first(p, pos);
                m[mt][x] = -INFINITY;
                l[mt][x] = 0.f;
                const T *src = static_cast<const T *>(p.a.q) + (long long)(t.row + j) * p.a.d.q_stride[0] +
                               (long long)(kvh * p.group + h0 + g) * p.a.d.q_stride[1];
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int c = 16 * k + 8 * y + 2 * (lane & 3);
                        uint32_t v = r < rows && c < D ? *reinterpret_cast<const uint32_t *>(src + c) : 0u;
                        if (p.sign != 1)
                            v = (v & keep) ^ flip;
                        if constexpr (kQSmem)
                            *reinterpret_cast<uint32_t *>(qs + r * kQStride + c * 2) = v;
                        else
                            q[mt][k][x + 2 * y] = v;
                    }
            }
        if (kQSmem)
            __syncwarp();
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[mt][n][i] = 0.f;
    }

    // scores of a unit's tokens and their weights; mask: the tokens read;
    // [all0, all1): tokens that every row sees
    __device__ __forceinline__ void scores(const AttnParams &p, char *slot_ptr, uint32_t mask, int tok0, int all0, int all1, int lane)
    {
        const int D = dim(p), stride = kRowBytes;
        const uint32_t slot = smem_addr(slot_ptr);
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[mt][n][i] = 0.f;
        // lanes 0-7, 8-15: tokens 0-7, first and second 16 bytes; 16-23, 24-31: tokens 8-15
        const uint32_t a = slot + ((lane & 7) + ((lane >> 4) << 3)) * stride + ((lane >> 3) & 1) * 16;
        // (query rows in shared memory) lanes 0-7, 8-15: rows 0-7, 8-15, first 16 bytes; 16-31: second
        const uint32_t qa = kQSmem ? smem_addr(qs) + ((lane & 7) + (((lane >> 3) & 1) << 3)) * kQStride + (lane >> 4) * 16 : 0;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            if (16 * k < D) {
                uint32_t qf[NM][4];
#pragma unroll
                for (int mt = 0; mt < NM; ++mt) {
                    if constexpr (kQSmem)
                        ldsm4(qa + mt * 16 * kQStride + k * 32, qf[mt]);
                    else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            qf[mt][i] = q[mt][k][i];
                    }
                }
#pragma unroll
                for (int h = 0; h < NT; ++h) {
                    uint32_t b[4];
                    ldsm4(a + h * 16 * stride + k * 32, b);
#pragma unroll
                    for (int mt = 0; mt < NM; ++mt) {
                        mma16816(s[mt][2 * h], qf[mt], b[0], b[1]);
                        mma16816(s[mt][2 * h + 1], qf[mt], b[2], b[3]);
                    }
                }
            }
        }
        constexpr uint32_t kAll = NT == 1 ? 0xffffu : 0xffffffffu;
        if (mask != kAll || tok0 < all0 || tok0 > all1 - kUnit) {
#pragma unroll
            for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tt = 8 * n + 2 * (lane & 3) + i, tok = tok0 + tt;
                    const bool there = (mask >> tt) & 1;
#pragma unroll
                    for (int mt = 0; mt < NM; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (!there || tok < lo[mt][x] || tok >= hi[mt][x])
                                s[mt][n][2 * x + i] = -INFINITY;
                }
        }
        // The running maximum moves only when a score is past it by more than kSlack
        // (weights are then at most 2^kSlack, which fp32 sums and rows bear): most
        // units need no exchange between lanes and no rescaling (a prompt of 8192
        // tokens 3.04 -> 2.77 ms; fp32, 8 rows, 218 -> 193 us).
        float top[NM][2];
        bool past = false;
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = s[mt][0][2 * x];
#pragma unroll
                for (int n = 0; n < 2 * NT; ++n)
                    v = fmaxf(v, fmaxf(s[mt][n][2 * x], s[mt][n][2 * x + 1]));
                top[mt][x] = v;
                past |= (v - m[mt][x]) * p.f > kSlack;
            }
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int mt = 0; mt < NM; ++mt) {
                float keep[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = fmaxf(top[mt][x], m[mt][x]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    keep[x] = exp2_fast((m[mt][x] - (v == -INFINITY ? 0.f : v)) * p.f);
                    m[mt][x] = v;
                    l[mt][x] *= keep[x];
                }
                if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[mt][n][i] *= keep[i >> 1];
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float base = m[mt][x] == -INFINITY ? 0.f : m[mt][x];
                const f32x2 less = pk2(-base, -base), ff = pk2(p.f, p.f);
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 2 * NT; ++n) {
                    float *v = &s[mt][n][2 * x];
                    const f32x2 e = mul2(add2(pk2(v[0], v[1]), less), ff);
                    v[0] = exp2_fast(lo2(e));
                    v[1] = exp2_fast(hi2(e));
                    sum += v[0];
                    sum += v[1];
                }
                l[mt][x] += sum;
            }
    }

    // whether the values of one of these tokens hold an infinity or NaN
    __device__ __forceinline__ bool not_finite(const AttnParams &p, const char *slot_ptr, uint32_t tokens, int lane)
    {
        constexpr int kSegs = DP / 8, kAtOnce = 32 / kSegs;
        const int c = lane % kSegs;
        uint32_t bad = 0;
        if (8 * c < dim(p)) {
#pragma unroll 4
            for (int r = lane / kSegs; r < kUnit; r += kAtOnce)
                if ((tokens >> r) & 1) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(slot_ptr + r * kRowBytes + c * 16);
                    // (an exponent of ones carries into the sign's place)
                    bad |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                           ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
                }
        }
        return __any_sync(0xffffffffu, (bad & 0x80008000u) != 0);
    }

    // Tokens that some rows of the tile see and others do not, with values that are
    // not finite, are added row by row, to those that see them, and then left out
    // of the product: there a weight 0 times an infinity or NaN of theirs would
    // reach every row.
    // (Unrolled over the tokens: a running token number would index the score
    // registers at run time and put them in local memory.)
    __device__ __forceinline__ void partial_tokens(const AttnParams &p, char *slot_ptr, uint32_t part, int tok0, int lane)
    {
        const int stride = kRowBytes;
        const uint32_t slot = smem_addr(slot_ptr);
#pragma unroll
        for (int tt = 0; tt < kUnit; ++tt) {
            if (!((part >> tt) & 1))
                continue;
            const uint32_t row = slot + tt * stride;
            float wgt[NM][2];
#pragma unroll
            for (int mt = 0; mt < NM; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float &own = s[mt][tt >> 3][2 * x + (tt & 1)];
                    const bool sees = tok0 + tt >= lo[mt][x] && tok0 + tt < hi[mt][x];
                    wgt[mt][x] = __shfl_sync(0xffffffffu, own, (lane & ~3) | ((tt & 7) >> 1));
                    if (!sees)
                        wgt[mt][x] = -1.f;
                    if ((lane & 3) == ((tt & 7) >> 1))
                        own = 0.f;
                }
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                if (8 * n < dim(p)) {
                    uint32_t v;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(row + 16 * n + 4 * (lane & 3)) : "memory");
#pragma unroll
                    for (int mt = 0; mt < NM; ++mt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (!(wgt[mt][x] < 0.f)) {
                                o[mt][n][2 * x] += wgt[mt][x] * __uint_as_float(v << 16);
                                o[mt][n][2 * x + 1] += wgt[mt][x] * __uint_as_float(v & 0xffff0000u);
                            }
                }
            }
            __syncwarp();
            for (int c = lane; c < p.seg; c += 32)
                *reinterpret_cast<uint4 *>(slot_ptr + tt * stride + c * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }

    __device__ __forceinline__ void values(const AttnParams &p, char *slot_ptr, uint32_t mask, int tok0, int all0, int all1, int lane)
    {
        const int D = dim(p), stride = kRowBytes;
        if (tok0 < all0 || tok0 > all1 - kUnit) {
            // bit tt: every row sees token tok0 + tt
            const int a0 = min(max(all0 - tok0, 0), kUnit), a1 = min(max(all1 - tok0, 0), kUnit);
            const uint32_t all = a1 > a0 ? (0xffffffffu >> (32 - a1)) & (0xffffffffu << a0) : 0u;
            const uint32_t part = mask & ~all;
            if (part && not_finite(p, slot_ptr, part, lane))
                partial_tokens(p, slot_ptr, part, tok0, lane);
        }
        // lanes 0-7, 8-15: tokens 0-7, 8-15 of the first 16 bytes; 16-31: of the second
        const uint32_t a = smem_addr(slot_ptr) + ((lane & 7) + (((lane >> 3) & 1) << 3)) * stride + (lane >> 4) * 16;
#pragma unroll
        for (int h = 0; h < NT; ++h) {
            uint32_t hi4[NM][4], lo4[NM][4];
#pragma unroll
            for (int mt = 0; mt < NM; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float u = s[mt][2 * h + n][2 * x], v = s[mt][2 * h + n][2 * x + 1];
                        const uint32_t w = pack_bf16(u, v);
                        hi4[mt][2 * n + x] = w;
                        lo4[mt][2 * n + x] = pack_bf16(u - __uint_as_float(w << 16), v - __uint_as_float(w & 0xffff0000u));
                    }
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
                if (16 * n < D) {
                    uint32_t b[4];
                    ldsm4t(a + h * 16 * stride + n * 32, b);
                    // (the second terms are 0 or of either sign: an infinite value times
                    // the first is the sum's, times the second it would undo that.  An
                    // instruction per fragment register: a prompt of 8192 tokens 2739 us,
                    // without 2749; groups of 16 with 5 tokens 264 and 260.  First terms
                    // cut off instead of rounded, so that the second ones are positive,
                    // cost as much and a bit.)
                    const uint32_t c[4] = {finite_bf16x2(b[0]), finite_bf16x2(b[1]), finite_bf16x2(b[2]), finite_bf16x2(b[3])};
#pragma unroll
                    for (int mt = 0; mt < NM; ++mt) {
                        mma16816(o[mt][2 * n], hi4[mt], b[0], b[1]);
                        mma16816(o[mt][2 * n + 1], hi4[mt], b[2], b[3]);
                        mma16816(o[mt][2 * n], lo4[mt], c[0], c[1]);
                        mma16816(o[mt][2 * n + 1], lo4[mt], c[2], c[3]);
                    }
                }
            }
        }
    }

    // the sums over the four lanes of a row; the rows' maxima and sums to shared memory
    __device__ __forceinline__ void end(const AttnParams &p, float *ml, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
                l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
                if ((lane & 3) == 0) {
                    const int r = mt * 16 + x * 8 + (lane >> 2);
                    ml[2 * r] = m[mt][x];
                    ml[2 * r + 1] = l[mt][x];
                }
            }
    }
    // The warp's rows as they are, without a join: `out(r, c, x, y)` takes elements
    // c, c + 1 of row r, scaled by `scale(m, l)`, and `stat(r, m, l)` the rows'
    // maxima (0 for a row that saw nothing) and sums.
    template <typename Scale, typename Out, typename Stat>
    __device__ __forceinline__ void finish(const AttnParams &p, int rows, int lane, Scale scale, Out out, Stat stat)
    {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = mt * 16 + x * 8 + (lane >> 2);
                float ll = l[mt][x];
                ll += __shfl_xor_sync(0xffffffffu, ll, 1);
                ll += __shfl_xor_sync(0xffffffffu, ll, 2);
                const float mm = m[mt][x] == -INFINITY ? 0.f : m[mt][x], f = scale(ll);
                if (r < rows) {
                    if ((lane & 3) == 0)
                        stat(r, mm, ll);
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n)
                        if (8 * n < dim(p))
                            out(r, 8 * n + 2 * (lane & 3), o[mt][n][2 * x] * f, o[mt][n][2 * x + 1] * f);
                }
            }
    }
    // m becomes the factor that brings the warp's rows to the warps' joint maximum
    __device__ __forceinline__ void rescale(const AttnParams &p, const float *ml, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                m[mt][x] = exp2_fast((m[mt][x] - joint_max<MR>(ml, mt * 16 + x * 8 + (lane >> 2))) * p.f);
    }
    // the scaled rows, written to or added to buf [MR][ds]
    template <bool ADD>
    __device__ __forceinline__ void put(const AttnParams &p, float *buf, int ds, int rows, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = mt * 16 + x * 8 + (lane >> 2);
                if (r < rows) {
                    const float f = m[mt][x];
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n) {
                        const int c = 8 * n + 2 * (lane & 3);
                        if (8 * n < dim(p)) {
                            float2 *at = reinterpret_cast<float2 *>(buf + r * ds + c);
                            float2 v = make_float2(o[mt][n][2 * x] * f, o[mt][n][2 * x + 1] * f);
                            if (ADD) {
                                const float2 u = *at;
                                v.x += u.x;
                                v.y += u.y;
                            }
                            *at = v;
                        }
                    }
                }
            }
    }
};

// ---- the arithmetic: fp32 ---------------------------------------------------

// Scores: a lane takes two tokens (half a unit apart) and a part of the head's
// elements, so that a query segment read from shared memory (the same for all
// lanes of a part) serves two tokens: those reads bound the scores of several
// rows.  The parts are added by shuffles, after which lane l has token l.
// Output: a lane holds 4 elements of every row (8 for heads above 128); for heads
// of at most 64 the half warps take tokens in turn.  The weights go through
// shared memory.  Products and sums are packed pairs of fp32 FMA.
template <int MRows, int DP, bool EX>
struct Simt {
    using T = float;
    static constexpr int MR = MRows, kDim = DP, kUnit = DP > 64 ? 16 : 32;
    static constexpr bool kExact = EX;
    static constexpr int kParts = 64 / kUnit;            // parts of the elements in the scores
    static constexpr int kGroups = DP <= 64 ? 2 : 1;     // tokens at a time in the output
    static constexpr int NV = (DP + 127) / 128;          // float4 of the output per lane and row
    f32x2 o[MR][NV][2];
    float m[MR], l[MR];   // m: the running maximum of q.k (of -q.k for a negative scale)
    int lo[MR], hi[MR];
    float *qs, *ps;       // the warp's query rows [MR][DP] and weights [MR][kUnit]
    static constexpr int kQBytes = MR * (DP + kUnit) * 4;   // per warp
    static constexpr bool kQSmem = false;

    __device__ __forceinline__ static int dim(const AttnParams &p) { return EX ? DP : p.a.d.headdim; }
    // of a ring slot: an odd number of segments, so that 8 rows' segments lie in different banks
    static constexpr int kRowBytes = (DP / 4 | 1) * 16;

    __device__ __forceinline__ void begin(const AttnParams &p, const Tile &t, int item, int lane)
    {
        const int kvh = p.nhb == 1 ? item : item / p.nhb, hb = item - kvh * p.nhb, D = dim(p);
        const int h0 = hb * p.gh, nh = min(p.gh, p.group - h0), rows = t.nq * nh;
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            const int rr = min(r, rows - 1), j = t.nq == 1 ? 0 : rr / nh, g = rr - j * nh;
            const int pos = p.a.positions[t.row + j];
            hi[r] = seen_end(p, pos);
            lo[r] = seen_first(p, pos);
            m[r] = -INFINITY;
            l[r] = 0.f;
            const float *src = static_cast<const float *>(p.a.q) + (long long)(t.row + j) * p.a.d.q_stride[0] +
                               (long long)(kvh * p.group + h0 + g) * p.a.d.q_stride[1];
            for (int c = 4 * lane; c < DP; c += 128) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < rows && c < D && p.sign != 0)
                    v = *reinterpret_cast<const float4 *>(src + c);
                if (p.sign < 0)
                    v = make_float4(-v.x, -v.y, -v.z, -v.w);
                *reinterpret_cast<float4 *>(qs + r * DP + c) = v;
            }
#pragma unroll
            for (int n = 0; n < NV; ++n)
                o[r][n][0] = o[r][n][1] = pk2(0.f, 0.f);
        }
        __syncwarp();
    }

    __device__ __forceinline__ void scores(const AttnParams &p, char *slot, uint32_t mask, int tok0, int all0, int all1, int lane)
    {
        constexpr int kHalf = kUnit / 2, NC = MR > 4 ? 1 : 2;   // NC: sums per row and token
        const int part = lane / kHalf, tt = lane % kUnit, D = dim(p);
        const ulonglong2 *k0 = reinterpret_cast<const ulonglong2 *>(slot + (lane % kHalf) * kRowBytes);
        const ulonglong2 *k1 = reinterpret_cast<const ulonglong2 *>(slot + (lane % kHalf + kHalf) * kRowBytes);
        f32x2 acc[MR][2][NC];
#pragma unroll
        for (int r = 0; r < MR; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    acc[r][t][i] = pk2(0.f, 0.f);
#pragma unroll 2
        for (int c = part; c < D / 4; c += kParts) {
            const ulonglong2 ka = k0[c], kb = k1[c];
#pragma unroll
            for (int r = 0; r < MR; ++r) {
                const ulonglong2 qv = *reinterpret_cast<const ulonglong2 *>(qs + r * DP + 4 * c);
                acc[r][0][0] = fma2(qv.x, ka.x, acc[r][0][0]);
                acc[r][1][0] = fma2(qv.x, kb.x, acc[r][1][0]);
                acc[r][0][NC - 1] = fma2(qv.y, ka.y, acc[r][0][NC - 1]);
                acc[r][1][NC - 1] = fma2(qv.y, kb.y, acc[r][1][NC - 1]);
            }
        }
        constexpr uint32_t kAll = kUnit == 16 ? 0xffffu : 0xffffffffu;
        const bool masked = mask != kAll || tok0 < all0 || tok0 > all1 - kUnit;
        float sc[MR];
        bool past = false;
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            float s0 = lo2(acc[r][0][0]) + hi2(acc[r][0][0]), s1 = lo2(acc[r][1][0]) + hi2(acc[r][1][0]);
            if (NC == 2) {
                s0 += lo2(acc[r][0][NC - 1]) + hi2(acc[r][0][NC - 1]);
                s1 += lo2(acc[r][1][NC - 1]) + hi2(acc[r][1][NC - 1]);
            }
            // neighbouring parts exchange: one keeps the first token, one the second
            float v = (part & 1 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, part & 1 ? s0 : s1, kHalf);
            if (kParts == 4)
                v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (masked && (!((mask >> tt) & 1) || tok0 + tt < lo[r] || tok0 + tt >= hi[r]))
                v = -INFINITY;
            sc[r] = v;
            past |= (v - m[r]) * p.f > kSlack;
        }
        if (__any_sync(0xffffffffu, past)) {   // (as for bf16)
#pragma unroll
            for (int r = 0; r < MR; ++r) {
                float top = fmaxf(sc[r], m[r]);
#pragma unroll
                for (int x = kUnit / 2; x >= 1; x >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float keep = exp2_fast((m[r] - (top == -INFINITY ? 0.f : top)) * p.f);
                m[r] = top;
                l[r] *= keep;
                if (keep != 1.f) {
                    const f32x2 kk = pk2(keep, keep);
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        o[r][n][0] = mul2(o[r][n][0], kk);
                        o[r][n][1] = mul2(o[r][n][1], kk);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            const float e = exp2_fast((sc[r] - (m[r] == -INFINITY ? 0.f : m[r])) * p.f);
            l[r] += lane < kUnit ? e : 0.f;   // summed over the lanes at the end
            if (lane < kUnit)
                ps[r * kUnit + tt] = e;
        }
        __syncwarp();
    }

    // RAGGED: some rows do not see all of the tokens; one that a row does not see is
    // skipped for it (tokens not read are zero in the slot, with weight 0)
    template <bool RAGGED>
    __device__ __forceinline__ void add_values(const AttnParams &p, const char *slot, int tok0, int lane)
    {
        constexpr int kTok = kUnit / kGroups;   // tokens of a half warp, or of the warp
        const int grp = kGroups == 2 ? lane >> 4 : 0, el = 4 * (kGroups == 2 ? lane & 15 : lane), stride = kRowBytes;
        const char *v0 = slot + grp * kTok * stride + 4 * el;
        const float *w0 = ps + grp * kTok;
#pragma unroll RAGGED ? 1 : 2
        for (int t4 = 0; t4 < kTok; t4 += 4) {
            float4 w[MR];
#pragma unroll
            for (int r = 0; r < MR; ++r)
                w[r] = *reinterpret_cast<const float4 *>(w0 + r * kUnit + t4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = tok0 + grp * kTok + t4 + i;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    ulonglong2 v = make_ulonglong2(0, 0);
                    if (EX || el + 128 * n < dim(p))
                        v = *reinterpret_cast<const ulonglong2 *>(v0 + (t4 + i) * stride + 512 * n);
#pragma unroll
                    for (int r = 0; r < MR; ++r) {
                        const float e = i == 0 ? w[r].x : i == 1 ? w[r].y : i == 2 ? w[r].z : w[r].w;
                        if (!RAGGED || (tok >= lo[r] && tok < hi[r])) {
                            o[r][n][0] = fma2(pk2(e, e), v.x, o[r][n][0]);
                            o[r][n][1] = fma2(pk2(e, e), v.y, o[r][n][1]);
                        }
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void values(const AttnParams &p, char *slot, uint32_t mask, int tok0, int all0, int all1, int lane)
    {
        if (tok0 < all0 || tok0 > all1 - kUnit)
            add_values<true>(p, slot, tok0, lane);
        else
            add_values<false>(p, slot, tok0, lane);
        __syncwarp();
    }

    __device__ __forceinline__ void add_groups()
    {
        if (kGroups == 2) {
#pragma unroll
            for (int r = 0; r < MR; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    o[r][0][i] = pk2(lo2(o[r][0][i]) + __shfl_xor_sync(0xffffffffu, lo2(o[r][0][i]), 16),
                                     hi2(o[r][0][i]) + __shfl_xor_sync(0xffffffffu, hi2(o[r][0][i]), 16));
        }
    }
    // as Mma's
    template <typename Scale, typename Out, typename Stat>
    __device__ __forceinline__ void finish(const AttnParams &p, int rows, int lane, Scale scale, Out out, Stat stat)
    {
        add_groups();
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            float ll = l[r];
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1)
                ll += __shfl_xor_sync(0xffffffffu, ll, x);
            const float mm = m[r] == -INFINITY ? 0.f : m[r], f = scale(ll);
            if (r < rows && (kGroups == 1 || lane < 16)) {
                if (lane == 0)
                    stat(r, mm, ll);
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = 4 * lane + 128 * n;
                    if (c < dim(p)) {
                        out(r, c, lo2(o[r][n][0]) * f, hi2(o[r][n][0]) * f);
                        out(r, c + 2, lo2(o[r][n][1]) * f, hi2(o[r][n][1]) * f);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void end(const AttnParams &p, float *ml, int lane)
    {
#pragma unroll
        for (int r = 0; r < MR; ++r) {
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1)
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
            if (lane == 0) {
                ml[2 * r] = m[r];
                ml[2 * r + 1] = l[r];
            }
        }
        add_groups();
    }
    __device__ __forceinline__ void rescale(const AttnParams &p, const float *ml, int)
    {
#pragma unroll
        for (int r = 0; r < MR; ++r)
            m[r] = exp2_fast((m[r] - joint_max<MR>(ml, r)) * p.f);
    }
    template <bool ADD>
    __device__ __forceinline__ void put(const AttnParams &p, float *buf, int ds, int rows, int lane)
    {
        if (kGroups == 2 && lane >= 16)
            return;
#pragma unroll
        for (int r = 0; r < MR; ++r) {
            if (r < rows) {
                const float f = m[r];
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = 4 * lane + 128 * n;
                    if (c < dim(p)) {
                        float4 *at = reinterpret_cast<float4 *>(buf + r * ds + c);
                        float4 v = make_float4(lo2(o[r][n][0]) * f, hi2(o[r][n][0]) * f, lo2(o[r][n][1]) * f, hi2(o[r][n][1]) * f);
                        if (ADD) {
                            const float4 u = *at;
                            v.x += u.x;
                            v.y += u.y;
                            v.z += u.z;
                            v.w += u.w;
                        }
                        *at = v;
                    }
                }
            }
        }
    }
};

__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) { *reinterpret_cast<uint32_t *>(p) = pack_bf16(x, y); }

// shared memory: the warps' rings, their query rows (and fp32 weights), two
// join buffers (in the query rows' place where those are bf16) -- all of whole
// 16-byte segments -- then maxima, sums and slot masks.  NH: halves in
// a warp's ring.
template <typename M, int NH, bool SOLO>
struct Layout {
    static constexpr int kQuery = kWarps * M::kQBytes;
    static constexpr int kSmall = (kWarps * M::MR * 2 + M::MR * 2 + kWarps * NH) * 4;
    static constexpr __host__ __device__ int join_stride(int D) { return D + 8; }
    static constexpr int kRing = kWarps * NH * M::kUnit * M::kRowBytes;
    static constexpr __host__ __device__ int join_bytes(int D) { return SOLO ? 0 : 2 * M::MR * join_stride(D) * 4; }
    static constexpr __host__ __device__ int middle_bytes(int D)
    {
        return M::kQSmem ? (kQuery > join_bytes(D) ? kQuery : join_bytes(D)) : kQuery + join_bytes(D);
    }
    static constexpr __host__ __device__ int total(int D) { return kRing + middle_bytes(D) + kSmall; }
};

// SOLO: shares of warps, for many tiles: a warp goes through whole tiles without
// a barrier, and a tile is cut into a few parts at most.  Else shares of CTAs,
// for few: a tile is then cut into many parts, and joining a CTA's warps first
// leaves a quarter of them to the second launch.
template <typename M, int NH, bool SOLO, bool ALIGNED, int MB>
__global__ void __launch_bounds__(kThreads, MB) ssd_paged_attn_kernel(const __grid_constant__ AttnParams p)
{
    using T = typename M::T;
    using L = Layout<M, NH, SOLO>;
    constexpr int UT = M::kUnit;
    extern __shared__ __align__(16) char smem[];
    __shared__ Found found[kWarps];
    __shared__ long long tmp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, D = M::dim(p);
    constexpr int stride = M::kRowBytes;
    constexpr int kOwn = SOLO ? kWarps : 1;   // shares of a CTA at a time
    const int first_share = SOLO ? blockIdx.x * kWarps + w : blockIdx.x;
    // The parameters' cache lines cost some hundred cycles each when first
    // touched: before the wait.
    {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < (int)sizeof(AttnParams) / 4; i += 16)
            x ^= reinterpret_cast<const uint32_t *>(&p)[i];
        asm volatile("" ::"r"(x));
    }
    constexpr int half_bytes = UT * stride;
    char *ring = smem + (size_t)w * NH * half_bytes;        // [NH][UT][stride]
    char *middle = smem + L::kRing;
    char *qs = middle + w * M::kQBytes;
    float *join = reinterpret_cast<float *>(middle + (M::kQSmem ? 0 : L::kQuery));   // (16-byte accesses up to here)
    float *ml = reinterpret_cast<float *>(middle + L::middle_bytes(D));   // [kWarps][MR][2]
    float *joint = ml + kWarps * M::MR * 2;                               // [MR] maxima, [MR] sums
    uint32_t *masks = reinterpret_cast<uint32_t *>(joint + M::MR * 2) + w * NH;
    const int ds = L::join_stride(D);
    // The call's launches are programmatic dependents: each starts while the one
    // before it runs out and waits here for all of it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Shares sh;
    Cursor cur;
    const bool few = p.few;
    const int padding = p.a.start ? p.a.start[p.a.d.nreq] : 0;   // first row of it
    if (few)
        sh = locate_few<UT, SOLO>(p, p.of_head == 1 ? 0 : div_fast(p.by_items, first_share), cur, reinterpret_cast<int4 *>(ring));
    else
        sh = locate<UT, SOLO>(p, reinterpret_cast<int *>(smem), tmp, found);
    // padding rows see nothing
    if (p.a.start) {
        const long long r0 = min((long long)max(padding, 0), (long long)p.a.d.nrows);
        for (long long i = r0 * p.a.d.nheads + blockIdx.x; i < p.a.d.nrows * p.a.d.nheads; i += gridDim.x) {
            const long long row = i / p.a.d.nheads, h = i - row * p.a.d.nheads;
            T *out = static_cast<T *>(p.a.out) + row * p.a.d.o_stride[0] + h * p.a.d.o_stride[1];
            for (int c = 4 * tid; c < D; c += 4 * kThreads)
                store4(out + c, make_float4(0.f, 0.f, 0.f, 0.f));
            if (p.a.lse && tid == 0)
                p.a.lse[i] = -INFINITY;
        }
        if (!SOLO)   // (there may be fewer tiles than the host could tell)
            for (long long i = sh.ntiles * p.items + blockIdx.x * kThreads + tid; i < p.ndesc; i += gridDim.x * kThreads)
                p.desc[i] = make_int4(-1, 0, 0, 0);
    }
    if (!few)
        __syncthreads();   // (the schedule's use of the ring's memory is over)
    // segments past the head's elements are read by the products: zero once
    if (!M::kExact) {
        for (int i = lane; i < NH * UT; i += 32)
            for (int c = p.seg; c * 16 < stride; ++c)
                *reinterpret_cast<uint4 *>(ring + (size_t)i * stride + c * 16) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();

    const int req0 = few ? cur.t.req : 0;   // (of more shares than one each, the first begins with the first tile)
    // Half h (K of unit h / 2, V when odd) goes to slot h % NH; at step h the half
    // h + NH - 1 is loaded: with an even ring V of a unit while K of one is used,
    // with an odd one K while K.  Every step is one group of asynchronous copies,
    // empty past the share's end.
    constexpr int step = SOLO ? 1 : kWarps;
    int head = 0, tail = 0;   // slots of the next half to load, to use
    // (one share each, but for more heads than there are warps or CTAs)
    for (int share = first_share; share < p.nshares; share += gridDim.x * kOwn) {
    const int j = div_fast(p.by_items, share), item = share - j * p.items;
    const long long u0 = p.of_head == 1 ? 0 : j * sh.per;
    if (SOLO && lane == 0)
        p.desc[share] = make_int4(-1, 0, 0, 0);
    if (u0 >= sh.total)   // (empty)
        continue;
    const int kvh = p.nhb == 1 ? item : item / p.nhb, hb = item - kvh * p.nhb;
    const int h0 = kvh * p.group + hb * p.gh, nh = min(p.gh, p.group - hb * p.gh);

    if (!few || share != first_share) {   // (a further share begins where its head does)
        const Found f = few ? Found{req0, 0, 0, 0} : found[SOLO ? w : 0];
        set_tile<UT>(p, cur.t, f.req, f.j);
        cur.tile = f.tile;
        cur.lin = f.lin;
    }
    const long long u1 = min(u0 + sh.per, sh.chunks ? cur.lin + cur.t.units : sh.total);
    Loader<T, M::kDim, M::kExact, ALIGNED, UT> ld;
    ld.c = cur;
    ld.u1 = u1;
    ld.set_head(p, kvh, lane);
    ld.set_tile_end(p);
    ld.u = (int)(u0 - cur.lin);
    ld.skip(p, SOLO ? 0 : w);
    ld.fetch_page(p, lane);
    auto load_k = [&]() {
        if (ld.u >= 0) {
            char *slot = ring + head * half_bytes;
            ld.offsets(p, lane);
            if (lane == 0)
                masks[head] = ld.mask;
            if constexpr (ALIGNED)
                ld.copy(p, ld.kb, ld.koff, p.ktok, smem_addr(slot), lane);
            else
                ld.copy_any(p, ld.kb, ld.koff[0], smem_addr(slot), lane);
            head = head + 1 == NH ? 0 : head + 1;
        }
        cp_commit();
    };
    auto load_v = [&]() {
        if (ld.u >= 0) {
            char *slot = ring + head * half_bytes;
            if constexpr (ALIGNED)
                ld.copy(p, ld.vb, ld.voff, p.vtok, smem_addr(slot), lane);
            else
                ld.copy_any(p, ld.vb, ld.voff[0], smem_addr(slot), lane);
            ld.skip(p, step);
            ld.fetch_page(p, lane);
            head = head + 1 == NH ? 0 : head + 1;
        }
        cp_commit();
    };
    M math;
    math.qs = reinterpret_cast<decltype(math.qs)>(qs);
    if constexpr (sizeof(T) == 4)
        math.ps = math.qs + M::MR * M::kDim;
    // tokens that every row of the tile sees: from the last row's first to the first row's last
    int all0, all1;
    auto begin = [&]() {
        all1 = seen_end(p, p.a.positions[cur.t.row]);
        all0 = seen_first(p, p.a.positions[cur.t.row + cur.t.nq - 1]);
        math.begin(p, cur.t, item, lane);
    };
    begin();   // (its loads are on their way beside the first table entry's)
#pragma unroll 1
    for (int i = 0; i < (NH - 1) / 2; ++i) {
        load_k();
        load_v();
    }
    if (NH % 2 == 0)
        load_k();

    int u = (int)(u0 - cur.lin);   // first unit of the share in this tile
    while (true) {
        const int ue = (int)min((long long)cur.t.units, u1 - cur.lin);   // the share's units of the tile: [u, ue)
        const int rows = cur.t.nq * nh;
        // this warp's units: all, or those whose number in the CTA's share is w modulo the warps
        const int skip = SOLO ? 0 : (w - (int)((cur.lin + u - u0) % kWarps) + kWarps) % kWarps;
        for (int x = u + skip; x < ue; x += step) {
            const int tok0 = (cur.t.ub + x) * UT;
            cp_wait<NH - 2>();
            __syncwarp();
            const uint32_t mask = masks[tail];
            if (NH % 2 == 0)
                load_v();
            else
                load_k();
            math.scores(p, ring + tail * half_bytes, mask, tok0, all0, all1, lane);
            tail = tail + 1 == NH ? 0 : tail + 1;
            cp_wait<NH - 2>();
            __syncwarp();
            if (NH % 2 == 0)
                load_k();
            else
                load_v();
            math.values(p, ring + tail * half_bytes, mask, tok0, all0, all1, lane);
            tail = tail + 1 == NH ? 0 : tail + 1;
        }
        const bool whole = u == 0 && ue == cur.t.units;
        const int slot = u > 0 ? 0 : 1;   // a tile begun in an earlier share, or in this one
        T *out = static_cast<T *>(p.a.out) + (long long)cur.t.row * p.a.d.o_stride[0] + (long long)h0 * p.a.d.o_stride[1];
        float *lse = p.a.lse ? p.a.lse + (long long)cur.t.row * p.a.d.nheads + h0 : nullptr;
        float *po = p.part_o + ((size_t)share * 2 + slot) * M::MR * D, *pml = p.part_ml + ((size_t)share * 2 + slot) * M::MR * 2;
        auto put_lse = [&](int r, float mm, float ll) {
            if (lse) {
                const int j = r / nh;
                lse[(long long)j * p.a.d.nheads + (r - j * nh)] = ll == 0.f ? -INFINITY : kLn2 * (mm * p.f + log2f(ll));
            }
        };
        if constexpr (SOLO) {
            if (whole)
                math.finish(p, rows, lane, [](float ll) { return ll == 0.f ? 0.f : 1.f / ll; },
                            [&](int r, int c, float a, float b) {
                                const int j = r / nh;
                                store2(out + (long long)j * p.a.d.o_stride[0] + (long long)(r - j * nh) * p.a.d.o_stride[1] + c, a, b);
                            }, put_lse);
            else
                math.finish(p, rows, lane, [](float) { return 1.f; },
                            [&](int r, int c, float a, float b) { store2(po + (size_t)r * D + c, a, b); },
                            [&](int r, float mm, float ll) { store2(pml + 2 * r, mm, ll); });
        } else {
            // join the warps: three barriers; the next tile's writes to ml, joint
            // and the buffers come after its own first or second one
            math.end(p, ml + w * M::MR * 2, lane);
            __syncthreads();
            if (tid < M::MR) {
                float ll = 0.f;
                const float base = joint_max<M::MR>(ml, tid);
#pragma unroll
                for (int i = 0; i < kWarps; ++i)
                    ll += ml[(i * M::MR + tid) * 2 + 1] * exp2_fast((ml[(i * M::MR + tid) * 2] - base) * p.f);
                joint[tid] = base;
                joint[M::MR + tid] = ll;
            }
            math.rescale(p, ml, lane);
            float *buf = join + (w & 1) * M::MR * ds;
            if (w >= 2)
                math.template put<false>(p, buf, ds, rows, lane);
            __syncthreads();
            if (w < 2)
                math.template put<true>(p, buf, ds, rows, lane);
            __syncthreads();
            const int n4 = D / 4;
            for (int i = tid; i < rows * n4; i += kThreads) {
                const int r = i / n4, c = 4 * (i - r * n4);
                const float4 x = *reinterpret_cast<const float4 *>(join + r * ds + c);
                const float4 y = *reinterpret_cast<const float4 *>(join + (M::MR + r) * ds + c);
                float4 v = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                const float ll = joint[M::MR + r];
                if (whole) {
                    const float inv = ll == 0.f ? 0.f : 1.f / ll;
                    const int j = r / nh;
                    v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
                    store4(out + (long long)j * p.a.d.o_stride[0] + (long long)(r - j * nh) * p.a.d.o_stride[1] + c, v);
                    if (c == 0)
                        put_lse(r, joint[r], ll);
                } else {
                    store4(po + (size_t)r * D + c, v);
                    if (c == 0)
                        store2(pml + 2 * r, joint[r], ll);
                }
            }
            if (M::kQSmem)
                __syncthreads();   // (the next tile's query rows go where the buffers are)
        }
        // where the parts of a cut tile are: this share and the head's next ones
        const long long at = SOLO ? share : (long long)cur.tile * p.items + item;
        // (a start array that descends has more tiles than there are entries)
        if ((SOLO ? !whole && slot == 1 && lane == 0 : slot == 1 && tid == 0) && at < p.ndesc)
            p.desc[at] = make_int4(whole ? -1 : cur.t.row, cur.t.nq | item << 8, (int)share,
                                   (int)div_units(cur.lin + cur.t.units - 1 - u0, sh.per) + 1);
        if (cur.lin + ue >= u1)
            break;
        u = 0;
        advance<UT>(p, cur);
        begin();
    }
    cp_wait<0>();
    __syncwarp();
    }
}

// Joins parts of row r of a cut tile: NW warps take parts in turn, lanes the
// elements, each warp in the running form, so that the parts' maxima and rows
// are loaded together, four at a time; then the warps through shared memory
// (sm, so: of the NW warps).
template <typename T, int MR, int NV, int NW>
__device__ __forceinline__ void join_row(const AttnParams &p, const int4 &d, int r, int w, int lane, float (*sm)[2], float (*so)[NV * 128])
{
    const int row = d.x, item = d.y >> 8, n = d.w, D = p.a.d.headdim;
    const int kvh = p.nhb == 1 ? item : item / p.nhb, hb = item - kvh * p.nhb, nh = min(p.gh, p.group - hb * p.gh);
    float mm = -INFINITY, ll = 0.f, o[NV][4] = {};
    // part i lies in the head's i-th share from d.z on: slot 1 of the first, slot 0 of the others
    for (int i = w; i < n; i += 4 * NW) {
        float pm[4], pl[4];
        float4 v[4][NV];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            pm[b] = -INFINITY;
            pl[b] = 0.f;
#pragma unroll
            for (int x = 0; x < NV; ++x)
                v[b][x] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int part = i + NW * b;
            if (part < n) {
                const size_t at = (((size_t)d.z + (size_t)part * p.items) * 2 + (part == 0 ? 1 : 0)) * MR + r;
                const float2 t = *reinterpret_cast<const float2 *>(p.part_ml + 2 * at);
                pm[b] = t.y == 0.f ? -INFINITY : t.x;   // (a part that saw nothing)
                pl[b] = t.y;
#pragma unroll
                for (int x = 0; x < NV; ++x)
                    if (4 * lane + 128 * x < D)
                        v[b][x] = *reinterpret_cast<const float4 *>(p.part_o + at * D + 4 * lane + 128 * x);
            }
        }
        const float mn = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), mm), base = mn == -INFINITY ? 0.f : mn;
        const float keep = exp2_fast((mm - base) * p.f);
        mm = mn;
        ll *= keep;
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[x][e] *= keep;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const float f = exp2_fast((pm[b] - base) * p.f);
            ll += pl[b] * f;
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                o[x][0] += f * v[b][x].x;
                o[x][1] += f * v[b][x].y;
                o[x][2] += f * v[b][x].z;
                o[x][3] += f * v[b][x].w;
            }
        }
    }
    float base = mm == -INFINITY ? 0.f : mm;
    if (NW > 1) {
#pragma unroll
        for (int x = 0; x < NV; ++x)
            *reinterpret_cast<float4 *>(&so[w][4 * lane + 128 * x]) = make_float4(o[x][0], o[x][1], o[x][2], o[x][3]);
        if (lane == 0) {
            sm[w][0] = mm;
            sm[w][1] = ll;
        }
        __syncthreads();
        if (w != 0)
            return;   // (the row is the first warp's)
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            top = fmaxf(top, sm[i][0]);
        base = top == -INFINITY ? 0.f : top;
        ll = 0.f;
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[x][e] = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float f = exp2_fast((sm[i][0] - base) * p.f);
            ll += sm[i][1] * f;
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(&so[i][4 * lane + 128 * x]);
                o[x][0] += f * v.x;
                o[x][1] += f * v.y;
                o[x][2] += f * v.z;
                o[x][3] += f * v.w;
            }
        }
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int j = (d.y & 0xff) == 1 ? 0 : r / nh, h = kvh * p.group + hb * p.gh + (r - j * nh);
    T *out = static_cast<T *>(p.a.out) + (long long)(row + j) * p.a.d.o_stride[0] + (long long)h * p.a.d.o_stride[1];
#pragma unroll
    for (int x = 0; x < NV; ++x)
        if (4 * lane + 128 * x < D)
            store4(out + 4 * lane + 128 * x, make_float4(o[x][0] * inv, o[x][1] * inv, o[x][2] * inv, o[x][3] * inv));
    if (p.a.lse && lane == 0)
        p.a.lse[(long long)(row + j) * p.a.d.nheads + h] = ll == 0.f ? -INFINITY : kLn2 * (base * p.f + log2f(ll));
}

__device__ __forceinline__ int desc_rows(const AttnParams &p, const int4 &d)
{
    const int hb = p.nhb == 1 ? 0 : (d.y >> 8) % p.nhb;
    return d.x < 0 ? 0 : (d.y & 0xff) * min(p.gh, p.group - hb * p.gh);
}

// Shares of a block of the join (where they are warps'): several only for tiles of a
// few rows, which leave the block's other warps idle (27 requests of 5 rows, window
// 665: 28 us with one share per block, 46 with four; fp32 tiles of one row, 576
// tiles: 51.5 with one, 50.1 with four).
template <int MR> constexpr int kJoinShares = MR >= 8 ? 1 : 4;

// NV: float4 of a row per lane.  SOLO: few parts, a warp per row.  Else many parts: a
// block per tile and row.
constexpr int kJoinWarps = 8;   // of a block
template <typename T, int MR, int NV, bool SOLO>
__global__ void __launch_bounds__(32 * kJoinWarps) ssd_paged_attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int NW = kJoinWarps;
    __shared__ float sm[NW][2];
    __shared__ __align__(16) float so[NW][NV * 128];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (SOLO) {
        int4 d[kJoinShares<MR>];
#pragma unroll
        for (int k = 0; k < kJoinShares<MR>; ++k) {
            const int i = blockIdx.x * kJoinShares<MR> + k;
            d[k] = i < p.ndesc ? p.desc[i] : make_int4(-1, 0, 0, 0);
        }
        int at = w;   // rows of all four, dealt to the warps; those of many parts are left to all of them
#pragma unroll
        for (int k = 0; k < kJoinShares<MR>; ++k) {
            const int rows = d[k].w > 16 ? 0 : desc_rows(p, d[k]);
            for (; at < rows; at += NW)
                join_row<T, MR, NV, 1>(p, d[k], at, 0, lane, sm, so);
            at -= rows;
        }
#pragma unroll 1
        for (int k = 0; k < kJoinShares<MR>; ++k) {
            const int4 t = k == 0 ? d[0] : k == 1 ? d[1 % kJoinShares<MR>] : k == 2 ? d[2 % kJoinShares<MR>] : d[3 % kJoinShares<MR>];
            const int rows = t.w > 16 ? desc_rows(p, t) : 0;
            for (int r = 0; r < rows; ++r) {
                join_row<T, MR, NV, NW>(p, t, r, w, lane, sm, so);
                __syncthreads();   // (the next row's sums go where these are)
            }
        }
    } else {
        const int4 d = p.desc[blockIdx.x];
        if ((int)blockIdx.y < desc_rows(p, d))
            join_row<T, MR, NV, NW>(p, d, blockIdx.y, w, lane, sm, so);
    }
}

// ---- host: one variant's launches ---------------------------------------------

constexpr int kSmemMost = (227 << 10) - 1024;   // dynamic, beside the kernel's few static bytes

template <typename M, int NH, bool SOLO, bool ALIGNED, int MB>
cudaError_t launch(AttnParams &p, void *workspace, cudaStream_t stream)
{
    using T = typename M::T;
    static_assert(Layout<M, NH, SOLO>::total(M::kDim) <= kSmemMost);
    const int D = p.a.d.headdim;
    const int smem = std::max(Layout<M, NH, SOLO>::total(D), p.a.start ? (int)(p.a.d.nreq + 1) * 4 : 0);
    auto kernel = ssd_paged_attn_kernel<M, NH, SOLO, ALIGNED, MB>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> regs{0};   // (the same for every device)
    cudaError_t e = allow_smem(kernel, kSmemMost, done);
    if (e != cudaSuccess)
        return e;
    int r = regs.load(std::memory_order_relaxed);
    if (r == 0) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess)
            return e;
        regs.store(r = (at.numRegs + 7) / 8 * 8, std::memory_order_relaxed);
    }
    // CTAs per SM by shared memory (1 KB of the system's each) and registers
    const int per_sm = std::max(1, std::min({kMaxPerSm, (228 << 10) / (smem + 1024 + 256), 65536 / (r * kThreads)}));
    const int grid = std::min(kMaxCtas, p.sms * per_sm);
    const int own = grid * (SOLO ? kWarps : 1);
    p.of_head = std::max(1, own / p.items);
    p.nshares = p.of_head * p.items;
    const size_t shares = (size_t)p.nshares;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = p.part_o + shares * 2 * M::MR * D;
    p.desc = reinterpret_cast<int4 *>(p.part_ml + shares * 2 * M::MR * 2);
    p.ndesc = SOLO ? (int)shares : (int)(most_tiles(p) * p.items);
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess)
        return e;
    note_launches(1);
    cfg.gridDim = SOLO ? dim3((p.ndesc + kJoinShares<M::MR> - 1) / kJoinShares<M::MR>) : dim3(p.ndesc, p.tok * p.gh);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, ssd_paged_attn_join_kernel<T, M::MR, (M::kDim + 127) / 128, SOLO>, p);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

// NH, NHS: halves in the ring with shares of CTAs, of warps; MB: CTAs per SM that the
// registers must leave room for with shares of warps.  Several CTAs per SM count for
// more than deep rings: heads of 128 with rings of 3 halves 181 us, of 2 172 (128
// requests of 1..4096 tokens); fp32 180 and 176 (32 requests of 100..8000).
template <typename M, int NH, int NHS, int MB, bool ALIGNED>
cudaError_t launch_shares(AttnParams &p, void *ws, cudaStream_t st)
{
    return solo_shares(p) ? launch<M, NHS, true, ALIGNED, MB>(p, ws, st) : launch<M, NH, false, ALIGNED, 1>(p, ws, st);
}

}  // namespace
}  // namespace ssd
