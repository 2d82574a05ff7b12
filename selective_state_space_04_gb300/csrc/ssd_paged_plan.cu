// ssd_paged_plan.cu -- block tables, positions and slots of one serving step,
// from the requests' lengths, without leaving the GPU.
//
// Three exclusive prefix sums over the requests (tokens brought, pages wanted,
// pages given back) decide everything: a request is granted iff its inclusive
// sums fit the step's rows and the free pages, so the granted ones are a prefix
// of those that bring tokens and fit their tables.  Every CTA of one cluster
// computes the sums for all requests itself (at most 8 requests per thread, one
// block scan) and keeps them in shared memory; then the CTAs share the writing:
// a page or token finds its request by binary search in those sums.  A new
// page's number is read from the ring, not back from block_table, so nothing
// written by the call is read by it, and the one cluster barrier, after every
// CTA has read lens and ring_pos, is what allows both to be updated in place.
#include <cuda_runtime.h>

#include <cstdint>

#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kPerThread = SSD_PLAN_MAX_REQUESTS / 1024;   // requests per thread at most

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

// pages of n >= 0 tokens (without the overflow of n + ps - 1)
__device__ __forceinline__ int pages_of(int n, int ps) { return n > 0 ? (n - 1) / ps + 1 : 0; }

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

__global__ void __launch_bounds__(1024) ssd_paged_plan_kernel(PlanArgs a)
{
    extern __shared__ int smem[];
    __shared__ long long warp_tot[3][32];
    __shared__ unsigned long long s_tok, s_pg;
    __shared__ int s_refused;
    const int n = a.nreq, tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int pad = (n + 4) & ~3;   // n + 1 entries, rounded up to 16 bytes
    PlanSmem s{smem, smem + pad, smem + 2 * pad, smem + 3 * pad};
    int rank = 0, ncta = 1;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
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
    const int per = (n + nthr - 1) / nthr, r0 = tid * per;
    long long tok = 0, pg = 0, bk = 0;
    int len[kPerThread], nw[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        const int r = r0 + j;
        len[j] = nw[j] = 0;
        if (j < per && r < n) {
            len[j] = max(a.lens[r], 0);
            nw[j] = a.new_lens[r];
            const int held = pages_of(len[j], ps);
            if (nw[j] < 0)
                bk += min(held, a.max_pages);
            else if ((long long)len[j] + nw[j] <= room) {
                tok += nw[j];
                pg += pages_of(len[j] + nw[j], ps) - held;
            }
        }
    }
    const long long itok = warp_inclusive(tok, lane), ipg = warp_inclusive(pg, lane), ibk = warp_inclusive(bk, lane);
    if (lane == 31) {
        warp_tot[0][warp] = itok;
        warp_tot[1][warp] = ipg;
        warp_tot[2][warp] = ibk;
    }
    __syncthreads();
    long long ctok = itok - tok, cpg = ipg - pg, cbk = ibk - bk, allbk = 0;
    for (int w = 0; w < nthr / 32; ++w) {
        if (w < warp) {
            ctok += warp_tot[0][w];
            cpg += warp_tot[1][w];
            cbk += warp_tot[2][w];
        }
        allbk += warp_tot[2][w];
    }
    long long top_tok = 0, top_pg = 0;
    int refused = 0;
    const long long tok0 = ctok, pg0 = cpg;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        if (j < per && r0 + j < n && nw[j] >= 0) {
            const bool fits = (long long)len[j] + nw[j] <= room;
            if (fits) {
                ctok += nw[j];
                cpg += pages_of(len[j] + nw[j], ps) - pages_of(len[j], ps);
            }
            if (nw[j] > 0) {
                if (fits && ctok <= a.max_tokens && cpg <= free_pages) {
                    top_tok = ctok;
                    top_pg = cpg;
                } else
                    ++refused;
            }
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
    for (int j = 0; j < kPerThread; ++j) {
        const int r = r0 + j;
        if (j < per && r < n) {
            s.start[r] = (int)min(ctok, (long long)total);
            s.page[r] = (int)min(cpg, (long long)taken);
            s.back[r] = (int)min(cbk, (long long)cap);
            s.len[r] = len[j];
            const int held = pages_of(len[j], ps);
            if (nw[j] < 0)
                cbk += min(held, a.max_pages);
            else if ((long long)len[j] + nw[j] <= room) {
                ctok += nw[j];
                cpg += pages_of(len[j] + nw[j], ps) - held;
            }
        }
    }
    if (tid == 0) {
        s.start[n] = total;
        s.page[n] = taken;
        s.back[n] = back;
    }
    // every CTA has read lens and ring_pos: both may be overwritten now
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    const int gtid = rank * nthr + tid, gthr = ncta * nthr;
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
    // pages drawn from the ring's head into their requests' tables
    for (int i = gtid; i < taken; i += gthr) {
        const int r = find(s.page, n, i);
        const long long at = (long long)head_at + i;
        a.table[(size_t)r * a.max_pages + pages_of(s.len[r], ps) + (i - s.page[r])] = a.ring[at < cap ? at : at - cap];
    }
    // pages given back, to its tail
    for (int i = gtid; i < back; i += gthr) {
        const int r = find(s.back, n, i);
        const long long at = (long long)tail_at + i;
        a.ring[at < cap ? at : at - cap] = a.table[(size_t)r * a.max_pages + (i - s.back[r])];
    }
    // the step's rows
    for (int t = gtid; t < a.max_tokens; t += gthr) {
        int pos = -1, r = -1;
        long long slot = -1;
        if (t < total) {
            r = find(s.start, n, t);
            pos = s.len[r] + (t - s.start[r]);
            const int p = pos / ps, held = pages_of(s.len[r], ps);
            const long long at = (long long)head_at + s.page[r] + (p - held);
            const int page = p < held ? a.table[(size_t)r * a.max_pages + p] : a.ring[at < cap ? at : at - cap];
            slot = (long long)page * ps + (pos - p * ps);
        }
        a.positions[t] = pos;
        a.token_req[t] = r;
        a.slots[t] = slot;
    }
}

}  // namespace

cudaError_t plan_launch(const PlanArgs &a, cudaStream_t stream)
{
    SSD_NVTX_RANGE("plan_launch");
    const int pad = (a.nreq + 4) & ~3;
    const size_t smem = (size_t)pad * 4 * sizeof(int);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(ssd_paged_plan_kernel, ((SSD_PLAN_MAX_REQUESTS + 4) & ~3) * 4 * (int)sizeof(int), done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 8;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(8);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, ssd_paged_plan_kernel, a);
    if (e == cudaSuccess)
        note_launches(1);
    return e;
}

}  // namespace ssd
