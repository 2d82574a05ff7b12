// ssd_paged_plan.cu -- block tables, positions and slots of one serving step,
// from the requests' lengths, without leaving the GPU.
//
// Three prefix sums over the requests (tokens brought, pages wanted, pages given
// back) decide everything: a request is granted iff its inclusive
// sums fit the step's rows and the free pages, so the granted ones are a prefix
// of those that bring tokens and fit their tables.  Every CTA
// computes the sums for all requests itself (at most 8 requests per thread, one
// block scan) and keeps them in shared memory; then the CTAs share the writing:
// a page, or four consecutive rows of the step, find their request by binary
// search in those sums.  A new page's number is read from the ring, not back
// from block_table, so nothing written by the call is read by it.  Only an update
// in place of lens or ring_pos has to wait until every CTA has read them: the CTAs
// are then one cluster (8 at most) with a barrier; else there may be as many as
// the rows need (2048 requests with 125000 rows: 11.6 us, in a cluster 19.1).
//
// Bound by latency: three dependent loads, two scans, the search and the stores
// (128 requests: 7.5 us, of which the launch some 2; the bytes would take 1 ns).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ssd_internal.h"

namespace ssd {
namespace {

struct PlanSmem {
    int *start, *page, *back, *len;   // [nreq+1] x3 (exclusive sums), [nreq]
};

__device__ __forceinline__ long long warp_inclusive(long long v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    return v;
}

// exact floor(n / d) for 0 <= n < 2^31: (n * mul) >> sh
struct FastDiv {
    uint32_t mul, sh;
    explicit FastDiv(int d = 1) : sh(31)
    {
        while ((1u << (sh - 31)) < (uint32_t)d)
            ++sh;
        mul = (uint32_t)((1ull << sh) / (uint32_t)d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> sh); }
};

// pages of n >= 0 tokens (without the overflow of n + page_size - 1)
__device__ __forceinline__ int pages_of(int n, const FastDiv &by) { return n > 0 ? by(n - 1) + 1 : 0; }

// the last r in [0, n) with sum[r] <= x (sum ascending, sum[0] <= x)
__device__ __forceinline__ int find(const int *sum, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// PER: requests per thread at most
template <int PER>
__global__ void __launch_bounds__(1024) ssd_paged_plan_kernel(PlanArgs a, FastDiv by, int barrier)
{
    extern __shared__ int smem[];
    __shared__ long long warp_tot[3][32];
    __shared__ unsigned long long s_tok, s_pg;
    __shared__ int s_refused;
    const int n = a.nreq, tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int pad = (n + 4) & ~3;   // n + 1 entries, rounded up to 16 bytes
    PlanSmem s{smem, smem + pad, smem + 2 * pad, smem + 3 * pad};
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long head = a.ring_pos[0], tail = a.ring_pos[1];
    long long free_pages = tail - head;
    free_pages = free_pages < 0 ? 0 : (free_pages > a.ring_size ? a.ring_size : free_pages);
    const int cap = a.ring_size, ps = a.page_size;
    const long long room = (long long)a.max_pages * ps;
    if (tid == 0) {
        s_tok = 0;
        s_pg = 0;
        s_refused = 0;
    }
    const int r0 = tid * PER;
    long long tok = 0, pg = 0, bk = 0;
    int len[PER], nw[PER], held[PER], more[PER];   // more: pages wanted (-1: does not fit its table), or given back
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int r = r0 + j;
        len[j] = nw[j] = held[j] = more[j] = 0;
        if (r < n) {
            len[j] = max(a.lens[r], 0);
            nw[j] = a.new_lens[r];
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        held[j] = pages_of(len[j], by);
        if (nw[j] < 0) {
            more[j] = min(held[j], a.max_pages);
            bk += more[j];
        } else if ((long long)len[j] + nw[j] <= room) {
            more[j] = pages_of(len[j] + nw[j], by) - held[j];
            tok += nw[j];
            pg += more[j];
        } else
            more[j] = -1;
    }
    const long long itok = warp_inclusive(tok, lane), ipg = warp_inclusive(pg, lane), ibk = warp_inclusive(bk, lane);
    if (lane == 31) {
        warp_tot[0][warp] = itok;
        warp_tot[1][warp] = ipg;
        warp_tot[2][warp] = ibk;
    }
    __syncthreads();
    // the warps' sums, scanned by every warp for itself
    const bool there = lane < nthr / 32;
    const long long wt = warp_inclusive(there ? warp_tot[0][lane] : 0, lane), wp = warp_inclusive(there ? warp_tot[1][lane] : 0, lane),
                    wb = warp_inclusive(there ? warp_tot[2][lane] : 0, lane);
    const int left = max(warp - 1, 0);
    const long long lt = __shfl_sync(0xffffffffu, wt, left), lp = __shfl_sync(0xffffffffu, wp, left),
                    lb = __shfl_sync(0xffffffffu, wb, left), allbk = __shfl_sync(0xffffffffu, wb, 31);
    long long ctok = itok - tok + (warp ? lt : 0), cpg = ipg - pg + (warp ? lp : 0), cbk = ibk - bk + (warp ? lb : 0);
    long long top_tok = 0, top_pg = 0;
    int refused = 0;
    const long long tok0 = ctok, pg0 = cpg;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (nw[j] > 0) {
            if (more[j] >= 0) {
                ctok += nw[j];
                cpg += more[j];
            }
            if (more[j] >= 0 && ctok <= a.max_tokens && cpg <= free_pages) {
                top_tok = ctok;
                top_pg = cpg;
            } else
                ++refused;
        }
    }
    if (top_tok > 0) {
        atomicMax(&s_tok, (unsigned long long)top_tok);
        atomicMax(&s_pg, (unsigned long long)top_pg);
    }
    if (refused)
        atomicAdd(&s_refused, refused);
    __syncthreads();
    const int total = (int)s_tok, taken = (int)s_pg;   // (at most max_tokens and ring_size)
    const int back = (int)(allbk < cap ? allbk : cap);
    // the exclusive sums per request, cut off at what was granted
    ctok = tok0;
    cpg = pg0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int r = r0 + j;
        if (r < n) {
            s.start[r] = (int)min(ctok, (long long)total);
            s.page[r] = (int)min(cpg, (long long)taken);
            s.back[r] = (int)min(cbk, (long long)cap);
            s.len[r] = len[j];
            if (nw[j] < 0)
                cbk += more[j];
            else if (more[j] >= 0) {
                ctok += nw[j];
                cpg += more[j];
            }
        }
    }
    if (tid == 0) {
        s.start[n] = total;
        s.page[n] = taken;
        s.back[n] = back;
    }
    __syncthreads();
    if (barrier)   // every CTA has read lens and ring_pos: both may be overwritten now
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    const int gtid = blockIdx.x * nthr + tid, gthr = gridDim.x * nthr;
    // per request
    for (int r = gtid; r <= n; r += gthr) {
        a.start[r] = s.start[r];
        if (r < n) {
            const int got = s.start[r + 1] - s.start[r];
            a.granted[r] = got;
            a.lens_out[r] = a.new_lens[r] < 0 ? 0 : s.len[r] + got;
        }
    }
    if (gtid == 0) {
        a.ring_pos_out[0] = head + taken;
        a.ring_pos_out[1] = tail + back;
        a.counts[0] = total;
        a.counts[1] = taken;
        a.counts[2] = back;
        a.counts[3] = s_refused;
    }
    int head_at = (int)(head % cap), tail_at = (int)(tail % cap);
    head_at += head_at < 0 ? cap : 0;
    tail_at += tail_at < 0 ? cap : 0;
    // pages drawn from the ring's head into their requests' tables, and pages given
    // back to its tail: several per thread at once, so that their loads overlap
    constexpr int kBatch = 4;
    for (long long i0 = gtid; i0 < taken; i0 += (long long)kBatch * gthr) {
        int page[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long i = i0 + (long long)k * gthr, at = head_at + i;
            if (i < taken)
                page[k] = a.ring[at < cap ? at : at - cap];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long i = i0 + (long long)k * gthr;
            if (i < taken) {
                const int r = find(s.page, n, (int)i);
                a.table[(size_t)r * a.max_pages + pages_of(s.len[r], by) + (i - s.page[r])] = page[k];
            }
        }
    }
    for (long long i0 = gtid; i0 < back; i0 += (long long)kBatch * gthr) {
        int page[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long i = i0 + (long long)k * gthr;
            if (i < back) {
                const int r = find(s.back, n, (int)i);
                page[k] = a.table[(size_t)r * a.max_pages + (i - s.back[r])];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long i = i0 + (long long)k * gthr, at = tail_at + i;
            if (i < back)
                a.ring[at < cap ? at : at - cap] = page[k];
        }
    }
    // the step's rows, four at a time
    for (long long t0 = 4ll * gtid; t0 < a.max_tokens; t0 += 4ll * gthr) {
        int r = -1, page = -1, off = 0, p = 0, held = 0, end = 0, pos = 0;
        int positions[4], reqs[4];
        long long slots[4];
        auto fetch_page = [&]() {
            const long long at = (long long)head_at + s.page[r] + (p - held);
            page = p < held ? a.table[(size_t)r * a.max_pages + p] : a.ring[at < cap ? at : at - cap];
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (int)t0 + i;
            positions[i] = reqs[i] = -1;
            slots[i] = -1;
            if (t >= total)
                continue;
            if (t >= end) {   // the row's request (the last that starts at or before it)
                if (i == 0)
                    r = find(s.start, n, t);
                else
                    while (s.start[r + 1] <= t)
                        ++r;
                end = s.start[r + 1];
                held = pages_of(s.len[r], by);
                pos = s.len[r] + (t - s.start[r]);
                p = by(pos);
                off = pos - p * ps;
                fetch_page();
            } else {
                ++pos;
                if (++off == ps) {
                    off = 0;
                    ++p;
                    fetch_page();
                }
            }
            positions[i] = pos;
            reqs[i] = r;
            slots[i] = (long long)page * ps + off;
        }
        if (t0 + 4 <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(positions[0], positions[1], positions[2], positions[3]);
            *reinterpret_cast<int4 *>(a.token_req + t0) = make_int4(reqs[0], reqs[1], reqs[2], reqs[3]);
            *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(slots[0], slots[1]);
            *reinterpret_cast<longlong2 *>(a.slots + t0 + 2) = make_longlong2(slots[2], slots[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < a.max_tokens) {
                    a.positions[t0 + i] = positions[i];
                    a.token_req[t0 + i] = reqs[i];
                    a.slots[t0 + i] = slots[i];
                }
        }
    }
}

}  // namespace

namespace {

template <int PER>
cudaError_t launch(const PlanArgs &a, int threads, cudaStream_t stream)
{
    const int pad = (a.nreq + 4) & ~3;
    const size_t smem = (size_t)pad * 4 * sizeof(int);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(ssd_paged_plan_kernel<PER>, ((SSD_PLAN_MAX_REQUESTS + 4) & ~3) * 4 * (int)sizeof(int), done);
    if (e != cudaSuccess)
        return e;
    // CTAs for the rows of the step, and for the pages that 32 requests may give back
    const bool in_place = a.lens_out == a.lens || a.ring_pos_out == a.ring_pos;
    const long long rows = ((long long)a.max_tokens + 4 * threads - 1) / (4 * threads), pages = (a.nreq + 31) / 32;
    int ctas = (int)std::min<long long>(std::max(std::max(rows, pages), 1ll), in_place ? 8 : sm_count());
    if (in_place)   // cluster sizes
        ctas = ctas > 4 ? 8 : ctas > 2 ? 4 : ctas;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = in_place && ctas > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, ssd_paged_plan_kernel<PER>, a, FastDiv(a.page_size), in_place && ctas > 1 ? 1 : 0);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace

cudaError_t plan_launch(const PlanArgs &a, cudaStream_t stream)
{
    SSD_NVTX_RANGE("plan_launch");
    // A request per thread as far as 1024 go (1000: 8.1 us, eight per thread 9.3;
    // 128: 7.5 and 10.1), then two (1500: 9.1 and 10.2), then eight with as many
    // threads as that takes (3000: 11.3, with 1024 threads 13.9).
    if (a.nreq <= 1024)
        return launch<1>(a, a.nreq <= 256 ? 256 : a.nreq <= 512 ? 512 : 1024, stream);
    return a.nreq <= 2048 ? launch<2>(a, 1024, stream) : launch<8>(a, (a.nreq + 255) / 256 * 32, stream);
}

}  // namespace ssd
