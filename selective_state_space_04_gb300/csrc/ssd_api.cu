// ssd_api.cu -- the C ABI of libssd: validation, path choice, scratch memory,
// launches.  Every entry point only enqueues on the caller's stream (except
// the host-buffer variant, which synchronises it at the end).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

std::atomic<uint64_t> g_launches{0};

size_t elem_size(int dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }

bool mul_ok(int64_t a, int64_t b, int64_t *out)
{
    if (a < 0 || b < 0)
        return false;
    if (a != 0 && b > INT64_MAX / a)
        return false;
    *out = a * b;
    return true;
}

struct Sizes {
    int64_t x, dt, bc, par, state;  // bytes
};

ssd_status_t check_dims(const ssd_dims_t *d, Sizes *sz)
{
    if (!d)
        return SSD_ERR_NULL_PTR;
    if (d->reserved != 0 || d->batch < 0 || d->seqlen < 0 || d->nheads < 1 || d->headdim < 1 ||
        d->dstate < 1 || d->ngroups < 1 || d->chunk < 1 || d->nheads % d->ngroups != 0)
        return SSD_ERR_INVALID_DIMS;
    if (d->dtype != SSD_DTYPE_F32 && d->dtype != SSD_DTYPE_BF16)
        return SSD_ERR_UNSUPPORTED_DTYPE;
    const uint32_t path = d->flags & SSD_PATH_MASK;
    if ((d->flags & ~(SSD_PATH_MASK | SSD_SCHEDULE_REQUEST_MASK | SSD_DIAG_STALL_HANDOFF)) != 0 ||
        path > SSD_PATH_DECODE)
        return SSD_ERR_INVALID_DIMS;
    int64_t bl, blh, t;
    const int64_t es = (int64_t)elem_size(d->dtype);
    if (!mul_ok(d->batch, d->seqlen, &bl) || !mul_ok(bl, d->nheads, &blh) ||
        !mul_ok(blh, d->headdim, &t) || !mul_ok(t, es, &sz->x) || !mul_ok(blh, 4, &sz->dt))
        return SSD_ERR_INVALID_DIMS;
    if (!mul_ok(bl, d->ngroups, &t) || !mul_ok(t, d->dstate, &t) || !mul_ok(t, es, &sz->bc))
        return SSD_ERR_INVALID_DIMS;
    sz->par = (int64_t)d->nheads * 4;
    if (!mul_ok(d->batch, d->nheads, &t) || !mul_ok(t, d->headdim, &t) ||
        !mul_ok(t, d->dstate, &t) || !mul_ok(t, 4, &sz->state))
        return SSD_ERR_INVALID_DIMS;
    if (sz->x > (INT64_C(1) << 46) || sz->state > (INT64_C(1) << 46) || d->seqlen >= (INT64_C(1) << 31))
        return SSD_ERR_INVALID_DIMS;
    return SSD_OK;
}

ScanArgs make_args(const void *x, const float *dt_raw, const float *dt_bias, const float *A_log,
                   const void *B, const void *C, const float *D, const float *init_state, void *y,
                   float *final_state, const ssd_dims_t *d)
{
    ScanArgs a;
    a.x = x;
    a.dt_raw = dt_raw;
    a.dt_bias = dt_bias;
    a.A_log = A_log;
    a.B = B;
    a.C = C;
    a.D = D;
    a.init_state = init_state;
    a.y = y;
    a.final_state = final_state;
    a.batch = d->batch;
    a.seqlen = d->seqlen;
    a.nheads = d->nheads;
    a.headdim = d->headdim;
    a.dstate = d->dstate;
    a.ngroups = d->ngroups;
    a.chunk = d->chunk;
    a.dtype = d->dtype;
    a.diag_stall = (d->flags & SSD_DIAG_STALL_HANDOFF) != 0;
    a.sched_req = (int)((d->flags & SSD_SCHEDULE_REQUEST_MASK) >> SSD_SCHEDULE_SHIFT);
    return a;
}

bool overlaps(const void *p, int64_t pn, const void *q, int64_t qn)
{
    if (!p || !q || pn <= 0 || qn <= 0)
        return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)qn && b < a + (uintptr_t)pn;
}

bool aligned16(const void *p) { return p == nullptr || ((uintptr_t)p & 15u) == 0; }

bool device_is_gb300_class()
{
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return false;
    return major == 10 && minor == 3;
}

// Why the chunked path refuses dims it does not support: its operands are bf16
// only, so another dtype is a dtype error; anything else is a shape error.
ssd_status_t chunk_refusal(const ScanArgs &a)
{
    return a.dtype != SSD_DTYPE_BF16 ? SSD_ERR_UNSUPPORTED_DTYPE : SSD_ERR_UNSUPPORTED;
}

// Unique id of the CUDA context current on this thread, or 0 when there is none
// or the driver cannot say.  The driver never reuses an id within a process, so
// the per-device caches below, keyed on it, notice a cudaDeviceReset or a
// re-created primary context and set themselves up again instead of handing out
// a pool, stream or address of a context that no longer exists.
uint64_t current_context_id()
{
    static std::once_flag once;
    static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
    static PFN_cuCtxGetId_v12000 get_id = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
        p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
    });
    CUcontext c = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&c) != CUDA_SUCCESS || !c || get_id(c, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// Resolves the path for validated dims.  Returns SSD_PATH_* or -status.
int32_t resolve_path(const ScanArgs &a, uint32_t requested, bool probe_device)
{
    const bool seq_ok = seq_supported(a.headdim, a.dstate);
    const bool decode_ok = decode_supported(a);
    if (requested == SSD_PATH_DECODE)
        return decode_ok ? (int32_t)SSD_PATH_DECODE : -(int32_t)SSD_ERR_UNSUPPORTED;
    if (requested == SSD_PATH_AUTO && decode_ok)
        return SSD_PATH_DECODE;
    const bool chunk_ok = chunk_supported(a) && (!probe_device || device_is_gb300_class());
    if (requested == SSD_PATH_SEQUENTIAL)
        return seq_ok ? (int32_t)SSD_PATH_SEQUENTIAL : -(int32_t)SSD_ERR_UNSUPPORTED;
    if (requested == SSD_PATH_CHUNKED)
        return chunk_ok ? (int32_t)SSD_PATH_CHUNKED : -(int32_t)chunk_refusal(a);
    if (chunk_ok)
        return SSD_PATH_CHUNKED;
    if (seq_ok)
        return SSD_PATH_SEQUENTIAL;
    return -(int32_t)SSD_ERR_UNSUPPORTED;
}

// Library-owned stream-ordered memory pool per device (kept cached so that
// repeated calls do not go back to the driver; set up again when the device's
// context has changed since).
cudaMemPool_t scratch_pool(int dev)
{
    static std::mutex mu;
    static cudaMemPool_t pools[64] = {};
    static uint64_t pool_ctx[64] = {};
    if (dev < 0 || dev >= 64)
        return nullptr;
    std::lock_guard<std::mutex> lk(mu);
    const uint64_t ctx = current_context_id();
    if (!pools[dev] || ctx == 0 || ctx != pool_ctx[dev]) {
        cudaMemPoolProps props;
        std::memset(&props, 0, sizeof(props));
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t p = nullptr;
        if (cudaMemPoolCreate(&p, &props) != cudaSuccess)
            return nullptr;
        uint64_t keep = UINT64_MAX;
        cudaMemPoolSetAttribute(p, cudaMemPoolAttrReleaseThreshold, &keep);
        pools[dev] = p;
        pool_ctx[dev] = current_context_id();   // the context exists now
    }
    return pools[dev];
}

// The host-buffer path pipelines pieces of whole batch rows through three
// library-owned streams per device (copies in, kernels, copies out).
constexpr int kHostPieces = 8;                          // most pieces per call
constexpr int64_t kHostPipelineMinBytes = 32ll << 20;   // smaller calls run as one piece

struct HostStreams {
    cudaStream_t in = nullptr, comp = nullptr, out = nullptr;
};

HostStreams host_streams(int dev)
{
    static std::mutex mu;
    static HostStreams streams[64];
    static uint64_t streams_ctx[64] = {};
    if (dev < 0 || dev >= 64)
        return HostStreams{};
    std::lock_guard<std::mutex> lk(mu);
    HostStreams &h = streams[dev];
    const uint64_t ctx = current_context_id();
    if (!h.in || ctx == 0 || ctx != streams_ctx[dev]) {
        HostStreams n;
        if (cudaStreamCreateWithFlags(&n.in, cudaStreamNonBlocking) != cudaSuccess ||
            cudaStreamCreateWithFlags(&n.comp, cudaStreamNonBlocking) != cudaSuccess ||
            cudaStreamCreateWithFlags(&n.out, cudaStreamNonBlocking) != cudaSuccess)
            return HostStreams{};
        h = n;
        streams_ctx[dev] = current_context_id();
    }
    return h;
}

// The paths that need no scratch: the sequential scan and the decode step.
ssd_status_t launch_direct(const ScanArgs &a, int32_t path, cudaStream_t st)
{
    const cudaError_t e = path == SSD_PATH_DECODE ? decode_launch(a, st) : seq_launch(a, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t run_device(const ScanArgs &a, uint32_t requested, cudaStream_t st)
{
    const int32_t path = resolve_path(a, requested, true);
    if (path < 0)
        return (ssd_status_t)(-path);
    if (path != SSD_PATH_CHUNKED)
        return launch_direct(a, path, st);
    const size_t ws_bytes = chunk_workspace_bytes(a);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    if (!pool)
        return SSD_ERR_CUDA;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, ws_bytes, pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    const ssd_status_t s = chunk_launch(a, ws, st);
    if (cudaFreeAsync(ws, st) != cudaSuccess && s == SSD_OK)
        return SSD_ERR_CUDA;
    return s;
}

ssd_status_t validate(const void *x, const float *dt_raw, const float *dt_bias, const float *A_log,
                      const void *B, const void *C, const float *D, const float *init_state,
                      const void *y, const float *final_state, const ssd_dims_t *dims, Sizes *sz)
{
    ssd_status_t s = check_dims(dims, sz);
    if (s != SSD_OK)
        return s;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!x || !dt_raw || !dt_bias || !A_log || !B || !C || !D || !y))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state};
    for (const void *p : ptrs)
        if (!aligned16(p))
            return SSD_ERR_MISALIGNED;
    if (work) {
        const void *ins[] = {x, dt_raw, dt_bias, A_log, B, C, D, init_state};
        const int64_t inb[] = {sz->x, sz->dt, sz->par, sz->par, sz->bc, sz->bc, sz->par, sz->state};
        for (int i = 0; i < 8; ++i) {
            if (overlaps(y, sz->x, ins[i], inb[i]))
                return SSD_ERR_ALIASING;
            if (overlaps(final_state, sz->state, ins[i], inb[i]) && !(i == 7 && final_state == init_state))
                return SSD_ERR_ALIASING;
        }
        if (overlaps(final_state, sz->state, y, sz->x))
            return SSD_ERR_ALIASING;
    } else if (init_state && final_state && init_state != final_state &&
               overlaps(final_state, sz->state, init_state, sz->state)) {
        return SSD_ERR_ALIASING;
    }
    return SSD_OK;
}

// ---- allocation-free variant of the chunked path ------------------------
//
// Some callers cannot let a library allocate device memory during a call:
// processes that reserve the whole device up front in an arena of their own
// (a serving stack that sizes weights, caches and activations at start-up)
// leave a library pool nothing to grow into, so a first-call allocation fails
// with out-of-memory; and drivers or virtualised devices without stream-ordered
// memory pools (cudaDevAttrMemoryPoolsSupported == 0) cannot serve
// cudaMallocFromPoolAsync at all.  For them ssd_scan_fwd_noalloc runs the
// chunked kernel with its scratch (abort word, handoff flags, chunk-handoff
// states) in this fixed module-scope array instead of a pool allocation.
//
// Limit: 32 MiB.  The kernel needs 256 B for the abort word, 64 B of flags
// per unit, and, when a batch-row x head-pair chain is split into several
// units, 64 KiB of handoff state per chain: about 20 MiB for batch 8 x 80
// heads at L = 4096, so roughly 500 split chains fit.  Larger needs are
// rejected with SSD_ERR_SCRATCH_LIMIT before anything is enqueued.
//
// Nothing in the array has to start at zero: every flag and the abort word
// are compared against a per-call tag that is never zero and never repeats
// within a process, so values left by an earlier call never match.
//
// The array is one per device and shared by every call: two calls whose
// kernels overlap in time on the same device (different streams, or threads
// without ordering between them) race on it and give wrong results or
// time out.  Calls ordered on one stream are safe.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of g_noalloc_scratch on the current device (the host-side name
// of the array is not a device address).  Looked up with that device current on
// the first call, and again whenever the device's context has changed since (a
// cudaDeviceReset unloads the module, and the array may come back elsewhere);
// cached otherwise.  Null on failure.
void *noalloc_scratch(int dev)
{
    static std::mutex mu;
    static void *addr[64] = {};
    static uint64_t addr_ctx[64] = {};
    if (dev < 0 || dev >= 64)
        return nullptr;
    std::lock_guard<std::mutex> lk(mu);
    const uint64_t ctx = current_context_id();
    if (!addr[dev] || ctx == 0 || ctx != addr_ctx[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) {
            addr[dev] = nullptr;
            return nullptr;
        }
        addr[dev] = p;
        addr_ctx[dev] = current_context_id();   // the lookup made the context current
    }
    return addr[dev];
}

// ---- strided operands of the attention-layer entry points ----------------

// [n0, n1, D] with strides in bytes, D contiguous
struct Strided {
    const void *p;
    int64_t n0, n1, s0, s1, width;   // counts, byte strides, bytes of one [D] row
    int64_t extent() const { return n0 > 0 && n1 > 0 ? (n0 - 1) * s0 + (n1 - 1) * s1 + width : 0; }
};

// Rows of `width` bytes at every combination of places on three axes.
struct Rows {
    const void *p;
    int64_t width;
    int64_t count[3], stride[3];   // strides >= 0, in bytes
};

struct StepAxis {
    int64_t stride, lo, hi;   // steps d with lo <= d <= hi
};

int64_t div_down(int64_t a, int64_t b) { return a / b - (a % b < 0); }   // b > 0

// Whether steps d exist, some of them not 0 unless `moved`, for which
// lo < sum of d * stride < hi.  Axes by falling strides: where each is longer than
// all after it together, two or three d per axis are in question.  `budget`: how
// many places to look at before taking it that there are such steps.
bool steps_between(const StepAxis *x, int n, int64_t lo, int64_t hi, bool moved, int &budget)
{
    if (--budget < 0)
        return true;
    if (n == 0)
        return moved && lo < 0 && hi > 0;
    int64_t least = 0, most = 0;   // what the axes after this one add
    for (int i = 1; i < n; ++i) {
        least += x[i].lo * x[i].stride;
        most += x[i].hi * x[i].stride;
    }
    const int64_t s = x[0].stride, from = std::max(x[0].lo, div_down(lo - most, s) + 1),
                  to = std::min(x[0].hi, -div_down(least - hi, s) - 1);
    for (int64_t d = from; d <= to; ++d)
        if (steps_between(x + 1, n - 1, lo - d * s, hi - d * s, moved || d != 0, budget))
            return true;
    return false;
}

constexpr int kViewBudget = 4096;

// whether two sets of rows share bytes
bool overlaps(const Rows &a, const Rows &b)
{
    StepAxis x[6];
    int n = 0;
    bool used[3] = {};
    if (!a.p || !b.p)
        return false;
    for (int i = 0; i < 3; ++i)
        if (a.count[i] <= 0 || b.count[i] <= 0)
            return false;
    for (int i = 0; i < 3; ++i) {
        if (a.count[i] <= 1 || a.stride[i] == 0)
            continue;
        StepAxis &t = x[n++] = {a.stride[i], 0, a.count[i] - 1};
        for (int j = 0; j < 3; ++j)
            if (!used[j] && b.count[j] > 1 && b.stride[j] == a.stride[i]) {
                used[j] = true;
                t.lo = 1 - b.count[j];
                break;
            }
    }
    for (int j = 0; j < 3; ++j)
        if (!used[j] && b.count[j] > 1 && b.stride[j] != 0)
            x[n++] = {b.stride[j], 1 - b.count[j], 0};
    std::sort(x, x + n, [](const StepAxis &u, const StepAxis &v) { return u.stride > v.stride; });
    const int64_t delta = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    int budget = kViewBudget;
    return steps_between(x, n, delta - a.width, delta + b.width, true, budget);
}

// whether the rows are all distinct memory
bool distinct_rows(const Rows &a)
{
    StepAxis x[3];
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (a.count[i] <= 0)
            return true;
        if (a.count[i] > 1) {
            if (a.stride[i] == 0)
                return false;
            x[n++] = {a.stride[i], 1 - a.count[i], a.count[i] - 1};
        }
    }
    std::sort(x, x + n, [](const StepAxis &u, const StepAxis &v) { return u.stride > v.stride; });
    int budget = kViewBudget;
    return !a.p || !steps_between(x, n, -a.width, a.width, false, budget);
}

Rows rows_of(const Strided &a) { return {a.p, a.width, {a.n0, a.n1, 1}, {a.s0, a.s1, 0}}; }
bool overlaps(const Strided &a, const Strided &b) { return overlaps(rows_of(a), rows_of(b)); }
bool distinct_rows(const Strided &a) { return distinct_rows(rows_of(a)); }

bool same_view(const Strided &a, const Strided &b)
{
    return a.p == b.p && a.n0 == b.n0 && a.n1 == b.n1 && a.s0 == b.s0 && a.s1 == b.s1;
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// strides: >= 0, multiples of 16 bytes, and small enough that the extent fits
bool strides_ok(const int64_t *s, int n, const int64_t *counts, int64_t es, ssd_status_t *why)
{
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        int64_t t;
        if (counts[i] <= 1)   // (the stride of a single row is not used)
            continue;
        if (s[i] < 0 || !mul_ok(s[i], es, &t) || !mul_ok(t, counts[i], &t) ||
            (total += t) > (INT64_C(1) << 46)) {
            *why = SSD_ERR_INVALID_DIMS;
            return false;
        }
        if (s[i] * es % 16 != 0) {
            *why = SSD_ERR_MISALIGNED;
            return false;
        }
    }
    return true;
}

ssd_status_t check_qk_dims(const ssd_qk_dims_t *d, bool cache, bool bwd)
{
    if (!d)
        return SSD_ERR_NULL_PTR;
    if (d->ntokens < 0 || d->ntokens >= (INT64_C(1) << 31) || d->max_pos < 0 || d->max_pos >= (INT64_C(1) << 31) ||
        d->nheads_q < 1 || d->nheads_k < 1 || d->nheads_q > (1 << 20) || d->nheads_k > (1 << 20) || d->headdim < 1 ||
        d->rotary_dim < 0 || d->rotary_dim > d->headdim || !(d->eps >= 0.f) || (d->flags & ~SSD_ROPE_INTERLEAVED) != 0)
        return SSD_ERR_INVALID_DIMS;
    if (d->dtype != SSD_DTYPE_F32 && d->dtype != SSD_DTYPE_BF16)
        return SSD_ERR_UNSUPPORTED_DTYPE;
    if (d->headdim % 8 != 0 || d->headdim > 256 || d->rotary_dim % 16 != 0 ||
        d->ntokens * std::max(d->nheads_q, d->nheads_k) > (INT64_C(1) << 30))   // (rows are counted in 32 bits)
        return SSD_ERR_UNSUPPORTED;
    const int64_t es = (int64_t)elem_size(d->dtype);
    const int64_t nq[] = {d->ntokens, d->nheads_q}, nk[] = {d->ntokens, d->nheads_k};
    ssd_status_t why = SSD_OK;
    if (!strides_ok(d->q_stride, 2, nq, es, &why) || !strides_ok(d->k_stride, 2, nk, es, &why) ||
        !strides_ok(d->qo_stride, 2, nq, es, &why) || !strides_ok(d->ko_stride, 2, nk, es, &why))
        return why;
    if (bwd && (!strides_ok(d->dq_stride, 2, nq, es, &why) || !strides_ok(d->dk_stride, 2, nk, es, &why)))
        return why;
    if (cache) {
        if (d->page_size < 1 || d->npages < 0 || d->npages >= (INT64_C(1) << 31))
            return SSD_ERR_INVALID_DIMS;
        const int64_t nc[] = {d->npages, d->page_size, d->nheads_k};
        if (!strides_ok(d->v_stride, 2, nk, es, &why) || !strides_ok(d->kc_stride, 3, nc, es, &why) ||
            !strides_ok(d->vc_stride, 3, nc, es, &why))
            return why;
    }
    return SSD_OK;
}

Strided view(const void *p, int64_t n0, int64_t n1, const int64_t *s, int64_t width, int64_t es)
{
    return {p, n0, n1, s[0] * es, s[1] * es, width};
}

// bytes that a paged cache spans
int64_t cache_extent(int64_t npages, int64_t page, int64_t heads, const int64_t *s, int64_t D, int64_t es)
{
    return npages > 0 ? ((npages - 1) * s[0] + (page - 1) * s[1] + (heads - 1) * s[2] + D) * es : 0;
}

ssd_status_t check_attn_dims(const ssd_attn_dims_t *d)
{
    if (!d)
        return SSD_ERR_NULL_PTR;
    int64_t t;
    if (d->flags != 0 || d->reserved != 0 || d->nrows < 0 || d->nrows >= (INT64_C(1) << 31) || d->nreq < 0 ||
        d->nreq >= (INT64_C(1) << 31) || d->npages < 0 || d->npages >= (INT64_C(1) << 31) || d->nheads < 1 ||
        d->nheads > (1 << 20) || d->nkv < 1 || d->nheads % d->nkv != 0 || d->headdim < 1 || d->page_size < 1 ||
        d->max_pages < 1 || (int64_t)d->page_size * d->max_pages >= (INT64_C(1) << 31) || d->window < 0 ||
        !(d->scale == d->scale) || d->table_stride < 0 || !mul_ok(d->nreq, d->table_stride, &t) ||
        t > (INT64_C(1) << 44))
        return SSD_ERR_INVALID_DIMS;
    if (d->dtype != SSD_DTYPE_F32 && d->dtype != SSD_DTYPE_BF16)
        return SSD_ERR_UNSUPPORTED_DTYPE;
    if (d->headdim % 8 != 0 || d->headdim > 256)
        return SSD_ERR_UNSUPPORTED;
    const int64_t es = (int64_t)elem_size(d->dtype);
    const int64_t nq[] = {d->nrows, d->nheads}, nc[] = {d->npages, d->page_size, d->nkv};
    ssd_status_t why = SSD_OK;
    if (!strides_ok(d->q_stride, 2, nq, es, &why) || !strides_ok(d->o_stride, 2, nq, es, &why) ||
        !strides_ok(d->kc_stride, 3, nc, es, &why) || !strides_ok(d->vc_stride, 3, nc, es, &why))
        return why;
    for (int i = 0; i < 2; ++i)   // the kernels hold page and token strides as 32-bit counts of 16 bytes
        if (nc[i] > 1 && (d->kc_stride[i] * es / 16 >= (INT64_C(1) << 32) || d->vc_stride[i] * es / 16 >= (INT64_C(1) << 32)))
            return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Runs `launch` with the caller's workspace, or with one from the library pool.
template <typename F>
ssd_status_t with_workspace(void *workspace, uint64_t have, size_t need, cudaStream_t st, F launch)
{
    if (need == 0)
        return launch(nullptr) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (workspace) {
        if (have < need)
            return SSD_ERR_SCRATCH_LIMIT;
        return launch(workspace) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    void *ws = nullptr;
    if (!pool || cudaMallocFromPoolAsync(&ws, need, pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    ssd_status_t s = launch(ws) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (cudaFreeAsync(ws, st) != cudaSuccess && s == SSD_OK)
        s = SSD_ERR_CUDA;
    return s;
}

}  // namespace

int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 152;
    n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return 152;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

uint64_t context_id() { return current_context_id(); }

void note_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status_t ssd_scan_fwd(const void *x, const float *dt_raw, const float *dt_bias,
                          const float *A_log, const void *B, const void *C, const float *D,
                          const float *init_state, void *y, float *final_state,
                          const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_scan_fwd");
    Sizes sz;
    ssd_status_t s = validate(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims, &sz);
    if (s != SSD_OK)
        return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->batch == 0)
        return SSD_OK;
    if (dims->seqlen == 0) {
        // no steps: the final state is the initial state (zero when none)
        if (!final_state || sz.state == 0)
            return SSD_OK;
        cudaError_t e = init_state ? (init_state == final_state
                                          ? cudaSuccess
                                          : cudaMemcpyAsync(final_state, init_state, (size_t)sz.state,
                                                            cudaMemcpyDeviceToDevice, st))
                                   : cudaMemsetAsync(final_state, 0, (size_t)sz.state, st);
        return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    const ScanArgs a = make_args(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims);
    return run_device(a, dims->flags & SSD_PATH_MASK, st);
}

ssd_status_t ssd_scan_fwd_host(const void *x, const float *dt_raw, const float *dt_bias,
                               const float *A_log, const void *B, const void *C,
                               const float *D, const float *init_state, void *y,
                               float *final_state, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_scan_fwd_host");
    Sizes sz;
    ssd_status_t s = validate(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims, &sz);
    if (s != SSD_OK)
        return s;
    if (dims->batch == 0 || (dims->seqlen == 0 && !final_state))
        return SSD_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->seqlen == 0) {
        if (init_state)
            std::memmove(final_state, init_state, (size_t)sz.state);
        else
            std::memset(final_state, 0, (size_t)sz.state);
        return SSD_OK;
    }
    auto up = [](int64_t v) { return (v + 255) & ~(int64_t)255; };
    const int64_t off_x = 0, off_dt = off_x + up(sz.x), off_bias = off_dt + up(sz.dt),
                  off_alog = off_bias + up(sz.par), off_B = off_alog + up(sz.par),
                  off_C = off_B + up(sz.bc), off_D = off_C + up(sz.bc), off_h0 = off_D + up(sz.par),
                  off_y = off_h0 + (init_state ? up(sz.state) : 0),
                  off_hf = off_y + up(sz.x), total = off_hf + (final_state ? up(sz.state) : 0);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    const HostStreams hs = host_streams(dev);
    if (!pool || !hs.in)
        return SSD_ERR_CUDA;
    char *buf = nullptr;
    if (cudaMallocFromPoolAsync((void **)&buf, (size_t)total, pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;

    // Pieces of whole batch rows go through three streams: copies in, kernels,
    // copies out, so the two copy directions and the scan overlap.  All kernels
    // stay on one stream (the persistent chunked kernel never shares the GPU
    // with another of its launches).  Each piece takes the schedule the whole
    // batch would (ranges and pieces give the same bits; a batch that would
    // take the split schedule runs as one piece), so the result is bitwise the
    // one ssd_scan_fwd gives.
    const int64_t Bt = dims->batch;
    const ScanArgs whole = make_args(buf + off_x, (const float *)(buf + off_dt), (const float *)(buf + off_bias),
                                     (const float *)(buf + off_alog), buf + off_B, buf + off_C,
                                     (const float *)(buf + off_D),
                                     init_state ? (const float *)(buf + off_h0) : nullptr, buf + off_y,
                                     final_state ? (float *)(buf + off_hf) : nullptr, dims);
    const uint32_t req = dims->flags & SSD_PATH_MASK;
    const int32_t path = resolve_path(whole, req, true);
    if (path < 0) {
        cudaFreeAsync(buf, st);
        cudaStreamSynchronize(st);
        return (ssd_status_t)(-path);
    }
    int sched = path == SSD_PATH_CHUNKED ? chunk_schedule(whole) : SSD_SCHEDULE_NONE;
    int pieces = (int)std::min<int64_t>(Bt, kHostPieces);
    if (sched == SSD_SCHEDULE_SPLIT || total < kHostPipelineMinBytes)
        pieces = 1;
    const int64_t xr = sz.x / Bt, dtr = sz.dt / Bt, bcr = sz.bc / Bt, str = sz.state / Bt;   // bytes per row

    cudaEvent_t start = nullptr, in_done[kHostPieces] = {}, comp_done[kHostPieces] = {}, end_in = nullptr,
                end_comp = nullptr, end_out = nullptr;
    bool ok = cudaEventCreateWithFlags(&start, cudaEventDisableTiming) == cudaSuccess &&
              cudaEventCreateWithFlags(&end_in, cudaEventDisableTiming) == cudaSuccess &&
              cudaEventCreateWithFlags(&end_comp, cudaEventDisableTiming) == cudaSuccess &&
              cudaEventCreateWithFlags(&end_out, cudaEventDisableTiming) == cudaSuccess;
    for (int k = 0; ok && k < pieces; ++k)
        ok = cudaEventCreateWithFlags(&in_done[k], cudaEventDisableTiming) == cudaSuccess &&
             cudaEventCreateWithFlags(&comp_done[k], cudaEventDisableTiming) == cudaSuccess;
    ok = ok && cudaEventRecord(start, st) == cudaSuccess && cudaStreamWaitEvent(hs.in, start, 0) == cudaSuccess &&
         cudaStreamWaitEvent(hs.comp, start, 0) == cudaSuccess && cudaStreamWaitEvent(hs.out, start, 0) == cudaSuccess;
    auto h2d = [&](int64_t off, const void *src, int64_t n) {
        if (ok && src && n > 0)
            ok = cudaMemcpyAsync(buf + off, src, (size_t)n, cudaMemcpyHostToDevice, hs.in) == cudaSuccess;
    };
    auto d2h = [&](void *dst, int64_t off, int64_t n) {
        if (ok && dst && n > 0)
            ok = cudaMemcpyAsync(dst, buf + off, (size_t)n, cudaMemcpyDeviceToHost, hs.out) == cudaSuccess;
    };
    h2d(off_bias, dt_bias, sz.par);
    h2d(off_alog, A_log, sz.par);
    h2d(off_D, D, sz.par);
    ssd_status_t rs = ok ? SSD_OK : SSD_ERR_CUDA;
    int64_t b0 = 0;
    for (int k = 0; k < pieces && rs == SSD_OK; ++k) {
        const int64_t rows = Bt / pieces + (k < Bt % pieces ? 1 : 0);
        const char *hx = static_cast<const char *>(x), *hB = static_cast<const char *>(B);
        const char *hC = static_cast<const char *>(C);
        h2d(off_x + b0 * xr, hx + b0 * xr, rows * xr);
        h2d(off_dt + b0 * dtr, reinterpret_cast<const char *>(dt_raw) + b0 * dtr, rows * dtr);
        h2d(off_B + b0 * bcr, hB + b0 * bcr, rows * bcr);
        h2d(off_C + b0 * bcr, hC + b0 * bcr, rows * bcr);
        if (init_state)
            h2d(off_h0 + b0 * str, reinterpret_cast<const char *>(init_state) + b0 * str, rows * str);
        ok = ok && cudaEventRecord(in_done[k], hs.in) == cudaSuccess &&
             cudaStreamWaitEvent(hs.comp, in_done[k], 0) == cudaSuccess;
        if (!ok) {
            rs = SSD_ERR_CUDA;
            break;
        }
        ssd_dims_t pd = *dims;
        pd.batch = rows;
        if (pieces > 1 && sched != SSD_SCHEDULE_NONE)
            pd.flags = (pd.flags & ~SSD_SCHEDULE_REQUEST_MASK) | ((uint32_t)sched << SSD_SCHEDULE_SHIFT);
        const ScanArgs a = make_args(buf + off_x + b0 * xr, (const float *)(buf + off_dt + b0 * dtr),
                                     (const float *)(buf + off_bias), (const float *)(buf + off_alog),
                                     buf + off_B + b0 * bcr, buf + off_C + b0 * bcr, (const float *)(buf + off_D),
                                     init_state ? (const float *)(buf + off_h0 + b0 * str) : nullptr,
                                     buf + off_y + b0 * xr,
                                     final_state ? (float *)(buf + off_hf + b0 * str) : nullptr, &pd);
        rs = run_device(a, req, hs.comp);
        if (rs != SSD_OK)
            break;
        ok = cudaEventRecord(comp_done[k], hs.comp) == cudaSuccess &&
             cudaStreamWaitEvent(hs.out, comp_done[k], 0) == cudaSuccess;
        d2h(static_cast<char *>(y) + b0 * xr, off_y + b0 * xr, rows * xr);
        if (final_state)
            d2h(reinterpret_cast<char *>(final_state) + b0 * str, off_hf + b0 * str, rows * str);
        if (!ok)
            rs = SSD_ERR_CUDA;
        b0 += rows;
    }
    // join the worker streams back into the caller's stream before the buffer goes
    const bool joined = end_in && end_comp && end_out && cudaEventRecord(end_in, hs.in) == cudaSuccess &&
                        cudaEventRecord(end_comp, hs.comp) == cudaSuccess &&
                        cudaEventRecord(end_out, hs.out) == cudaSuccess &&
                        cudaStreamWaitEvent(st, end_in, 0) == cudaSuccess &&
                        cudaStreamWaitEvent(st, end_comp, 0) == cudaSuccess &&
                        cudaStreamWaitEvent(st, end_out, 0) == cudaSuccess;
    if (!joined) {   // fall back to waiting on the host
        cudaStreamSynchronize(hs.in);
        cudaStreamSynchronize(hs.comp);
        cudaStreamSynchronize(hs.out);
        if (rs == SSD_OK)
            rs = SSD_ERR_CUDA;
    }
    cudaFreeAsync(buf, st);
    if (cudaStreamSynchronize(st) != cudaSuccess && rs == SSD_OK)
        rs = SSD_ERR_CUDA;
    for (cudaEvent_t e : {start, end_in, end_comp, end_out})
        if (e)
            cudaEventDestroy(e);
    for (int k = 0; k < pieces; ++k) {
        if (in_done[k])
            cudaEventDestroy(in_done[k]);
        if (comp_done[k])
            cudaEventDestroy(comp_done[k]);
    }
    return rs;
}

ssd_status_t ssd_scan_fwd_noalloc(const void *x, const float *dt_raw, const float *dt_bias,
                                  const float *A_log, const void *B, const void *C,
                                  const float *D, const float *init_state, void *y,
                                  float *final_state, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_scan_fwd_noalloc");
    Sizes sz;
    ssd_status_t s = validate(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims, &sz);
    if (s != SSD_OK)
        return s;
    // empty work: ssd_scan_fwd launches nothing and allocates nothing here
    if (dims->batch == 0 || dims->seqlen == 0)
        return ssd_scan_fwd(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims,
                            stream);
    // the chunked kernel is the only path here: another explicit request is refused
    const uint32_t req = dims->flags & SSD_PATH_MASK;
    if (req != SSD_PATH_AUTO && req != SSD_PATH_CHUNKED)
        return SSD_ERR_UNSUPPORTED;
    ScanArgs a = make_args(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims);
    if (a.sched_req == SSD_SCHEDULE_SPLIT)
        return SSD_ERR_UNSUPPORTED;
    a.scratch_cap = kNoAllocScratchBytes;
    const int32_t path = resolve_path(a, SSD_PATH_CHUNKED, true);
    if (path < 0)
        return (ssd_status_t)(-path);
    if (chunk_workspace_bytes(a) > kNoAllocScratchBytes)
        return SSD_ERR_SCRATCH_LIMIT;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    void *ws = noalloc_scratch(dev);
    if (!ws)
        return SSD_ERR_CUDA;
    return chunk_launch(a, ws, static_cast<cudaStream_t>(stream));
}

ssd_status_t ssd_scan_fwd_workspace_size(const ssd_dims_t *dims, uint64_t *bytes)
{
    if (!bytes)
        return SSD_ERR_NULL_PTR;
    Sizes sz;
    const ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    *bytes = 0;
    if (dims->batch == 0 || dims->seqlen == 0)
        return SSD_OK;
    const ScanArgs a = make_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, dims);
    const int32_t path = resolve_path(a, dims->flags & SSD_PATH_MASK, true);
    if (path < 0)
        return (ssd_status_t)(-path);
    if (path == SSD_PATH_CHUNKED)
        *bytes = chunk_workspace_bytes(a);
    return SSD_OK;
}

ssd_status_t ssd_scan_fwd_ws(const void *x, const float *dt_raw, const float *dt_bias,
                             const float *A_log, const void *B, const void *C, const float *D,
                             const float *init_state, void *y, float *final_state, void *workspace,
                             uint64_t workspace_bytes, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_scan_fwd_ws");
    Sizes sz;
    ssd_status_t s = validate(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims, &sz);
    if (s != SSD_OK)
        return s;
    if (!aligned16(workspace))
        return SSD_ERR_MISALIGNED;
    if (workspace && workspace_bytes > 0) {
        const void *args[] = {x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state};
        const int64_t argb[] = {sz.x, sz.dt, sz.par, sz.par, sz.bc, sz.bc, sz.par, sz.state, sz.x, sz.state};
        const int64_t wb = workspace_bytes > (uint64_t)INT64_MAX ? INT64_MAX : (int64_t)workspace_bytes;
        for (int i = 0; i < 10; ++i)
            if (overlaps(workspace, wb, args[i], argb[i]))
                return SSD_ERR_ALIASING;
    }
    // empty work needs no scratch: ssd_scan_fwd allocates nothing here
    if (dims->batch == 0 || dims->seqlen == 0)
        return ssd_scan_fwd(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims,
                            stream);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const ScanArgs a = make_args(x, dt_raw, dt_bias, A_log, B, C, D, init_state, y, final_state, dims);
    const int32_t path = resolve_path(a, dims->flags & SSD_PATH_MASK, true);
    if (path < 0)
        return (ssd_status_t)(-path);
    if (path != SSD_PATH_CHUNKED)
        return launch_direct(a, path, st);
    const size_t need = chunk_workspace_bytes(a);
    if (workspace_bytes < need)
        return SSD_ERR_SCRATCH_LIMIT;
    if (!workspace)
        return SSD_ERR_NULL_PTR;
    return chunk_launch(a, workspace, st);
}

int32_t ssd_select_path(const ssd_dims_t *dims)
{
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return -(int32_t)s;
    const ScanArgs a = make_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, dims);
    return resolve_path(a, dims->flags & SSD_PATH_MASK, true);
}

int32_t ssd_launches_per_call(const ssd_dims_t *dims)
{
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return -(int32_t)s;
    if (dims->batch == 0 || dims->seqlen == 0)
        return 0;
    const ScanArgs a = make_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, dims);
    const int32_t path = resolve_path(a, dims->flags & SSD_PATH_MASK, true);
    if (path < 0)
        return path;
    return path == SSD_PATH_CHUNKED ? chunk_launches(a) : 1;
}

int32_t ssd_chunk_schedule(const ssd_dims_t *dims)
{
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return -(int32_t)s;
    if (dims->batch == 0 || dims->seqlen == 0)
        return SSD_SCHEDULE_NONE;
    const ScanArgs a = make_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, dims);
    const int32_t path = resolve_path(a, dims->flags & SSD_PATH_MASK, true);
    if (path < 0)
        return path;
    return path == SSD_PATH_CHUNKED ? chunk_schedule(a) : SSD_SCHEDULE_NONE;
}

uint64_t ssd_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

ssd_status_t ssd_get_device_error(void *stream, uint32_t *code)
{
    if (!code)
        return SSD_ERR_NULL_PTR;
    const ssd_status_t s = chunk_read_device_error(static_cast<cudaStream_t>(stream), code);
    if (s != SSD_OK)
        return s;
    uint32_t bwd = 0, cplx = 0;   // the backward's and the complex chunk form's kernels keep their own words
    ssd_status_t s2 = bwd_tc_read_device_error(&bwd);
    if (s2 == SSD_OK)
        s2 = complex_tc_read_device_error(&cplx);
    if (s2 != SSD_OK)
        return s2;
    if (*code == 0)
        *code = bwd ? bwd : cplx;
    return SSD_OK;
}

const char *ssd_status_string(ssd_status_t status)
{
    switch ((int32_t)status) {
    case SSD_OK: return "ok";
    case SSD_ERR_INVALID_DIMS: return "invalid dimensions";
    case SSD_ERR_NULL_PTR: return "required pointer is null";
    case SSD_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case SSD_ERR_UNSUPPORTED: return "dtype, shape or path not supported";
    case SSD_ERR_CUDA: return "CUDA call failed";
    case SSD_ERR_TIMEOUT: return "kernel exceeded a bounded wait";
    case SSD_ERR_ALIASING: return "output overlaps an input";
    case SSD_ERR_SCRATCH_LIMIT: return "scratch needed exceeds the buffer the call may use";
    case SSD_ERR_UNSUPPORTED_DTYPE: return "dtype not supported";
    default: return "unknown status";
    }
}

int32_t ssd_abi_version(void) { return SSD_ABI_VERSION; }

ssd_status_t ssd_complex_scan_fwd(const void *x, const float *dt_raw, const float *dt_bias, const float *A_polar,
                                  const void *B, const void *C, const float *D, const float *init_state, void *y,
                                  float *final_state, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_complex_scan_fwd");
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    if ((dims->flags & ~SSD_PATH_MASK) != 0)
        return SSD_ERR_INVALID_DIMS;
    const uint32_t path = dims->flags & SSD_PATH_MASK;
    if (path != SSD_PATH_AUTO && path != SSD_PATH_SEQUENTIAL && path != SSD_PATH_CHUNKED)
        return SSD_ERR_UNSUPPORTED;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!x || !dt_raw || !dt_bias || !A_polar || !B || !C || !D || !y))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {x, dt_raw, dt_bias, A_polar, B, C, D, init_state, y, final_state};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    // outputs overlap no input (the state may be updated in place) and not each other
    const void *ins[] = {x, dt_raw, dt_bias, A_polar, B, C, D, init_state};
    const int64_t inb[] = {sz.x, sz.dt, sz.par, 2 * sz.par, sz.bc, sz.bc, sz.par, sz.state};
    const void *outs[] = {work ? y : nullptr, final_state};
    const int64_t outb[] = {sz.x, sz.state};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 8; ++i)
            if (overlaps(outs[o], outb[o], ins[i], inb[i]) && !(o == 1 && ins[i] == init_state && outs[o] == init_state))
                return SSD_ERR_ALIASING;
    if (overlaps(outs[0], outb[0], outs[1], outb[1]))
        return SSD_ERR_ALIASING;
    ComplexArgs ca;
    ca.x = x;
    ca.B = B;
    ca.C = C;
    ca.dt_raw = dt_raw;
    ca.dt_bias = dt_bias;
    ca.A_polar = A_polar;
    ca.D = D;
    ca.init_state = init_state;
    ca.y = y;
    ca.final_state = final_state;
    ca.batch = dims->batch;
    ca.seqlen = dims->seqlen;
    ca.nheads = dims->nheads;
    ca.headdim = dims->headdim;
    ca.dstate = dims->dstate;
    ca.ngroups = dims->ngroups;
    ca.dtype = dims->dtype;
    // the chunk form on the tensor cores where it applies (auto) or is asked for
    const bool tc = path != SSD_PATH_SEQUENTIAL && complex_tc_supported(ca);
    if (path == SSD_PATH_CHUNKED && !tc)
        return SSD_ERR_UNSUPPORTED;
    if (!tc && !complex_supported(ca))
        return SSD_ERR_UNSUPPORTED;
    if (dims->batch == 0)
        return SSD_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->seqlen == 0) {   // no steps: the state passes through (zero when not given)
        if (!final_state || final_state == init_state)
            return SSD_OK;
        const cudaError_t e = init_state ? cudaMemcpyAsync(final_state, init_state, (size_t)sz.state,
                                                           cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(final_state, 0, (size_t)sz.state, st);
        return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    return (tc ? complex_tc_launch(ca, st) : complex_launch(ca, st)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_trap_scan_fwd(const void *v, const void *k, const void *q, const float *dt, const float *a,
                               const float *trap, const float *D, const float *h0, const void *k0,
                               const void *v0, void *y, float *h_final, void *k_final, void *v_final,
                               const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_trap_scan_fwd");
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    const uint32_t path = dims->flags & SSD_PATH_MASK;
    if ((dims->flags & ~(SSD_PATH_MASK | SSD_SCHEDULE_REQUEST_MASK)) != 0)
        return SSD_ERR_INVALID_DIMS;
    if (path != SSD_PATH_AUTO && path != SSD_PATH_SEQUENTIAL && path != SSD_PATH_CHUNKED)
        return SSD_ERR_UNSUPPORTED;
    const int64_t es = dims->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const int64_t kst = dims->batch * dims->nheads * dims->dstate * es;   // k_state bytes
    const int64_t vst = dims->batch * dims->nheads * dims->headdim * es;  // v_state bytes
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!v || !k || !q || !dt || !a || !trap || !D || !y))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {v, k, q, dt, a, trap, D, h0, k0, v0, y, h_final, k_final, v_final};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    // outputs overlap no input (each state may be updated in place) and no other output
    const void *ins[] = {v, k, q, dt, a, trap, D, h0, k0, v0};
    const int64_t inb[] = {sz.x, sz.bc, sz.bc, sz.dt, sz.dt, sz.dt, sz.par, sz.state, kst, vst};
    const void *outs[] = {work ? y : nullptr, h_final, k_final, v_final};
    const int64_t outb[] = {sz.x, sz.state, kst, vst};
    const void *same[] = {nullptr, h0, k0, v0};   // the input each output may replace exactly
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 10; ++i)
            if (overlaps(outs[o], outb[o], ins[i], inb[i]) && !(outs[o] == same[o] && ins[i] == same[o]))
                return SSD_ERR_ALIASING;
        for (int o2 = o + 1; o2 < 4; ++o2)
            if (overlaps(outs[o], outb[o], outs[o2], outb[o2]))
                return SSD_ERR_ALIASING;
    }
    if (dims->batch == 0)
        return SSD_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->seqlen == 0) {
        // no steps: every carried state passes through unchanged (zero when not given)
        const void *src[] = {h0, k0, v0};
        void *dst[] = {h_final, k_final, v_final};
        const int64_t nb[] = {sz.state, kst, vst};
        for (int i = 0; i < 3; ++i) {
            if (!dst[i] || nb[i] == 0 || src[i] == dst[i])
                continue;
            const cudaError_t e = src[i] ? cudaMemcpyAsync(dst[i], src[i], (size_t)nb[i], cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(dst[i], 0, (size_t)nb[i], st);
            if (e != cudaSuccess)
                return SSD_ERR_CUDA;
        }
        return SSD_OK;
    }
    TrapArgs ta;
    ta.v = v;
    ta.k = k;
    ta.q = q;
    ta.dt = dt;
    ta.a = a;
    ta.trap = trap;
    ta.D = D;
    ta.h0 = h0;
    ta.k0 = k0;
    ta.v0 = v0;
    ta.y = y;
    ta.h_final = h_final;
    ta.k_final = k_final;
    ta.v_final = v_final;
    ta.batch = dims->batch;
    ta.seqlen = dims->seqlen;
    ta.nheads = dims->nheads;
    ta.headdim = dims->headdim;
    ta.dstate = dims->dstate;
    ta.ngroups = dims->ngroups;
    ta.dtype = dims->dtype;
    // the chunked tcgen05 kernel in its trapezoidal mode, or the sequential kernel
    ScanArgs ca = make_args(v, nullptr, nullptr, nullptr, k, q, D, h0, y, h_final, dims);
    ca.trap = true;
    ca.tdt = dt;
    ca.ta = a;
    ca.ttrap = trap;
    ca.k0 = k0;
    ca.v0 = v0;
    const bool chunk_ok = chunk_supported(ca) && device_is_gb300_class();
    const bool seq_ok = trap_supported(ta);
    bool chunked;
    if (path == SSD_PATH_CHUNKED)
        chunked = true;
    else if (path == SSD_PATH_SEQUENTIAL)
        chunked = false;
    else   // one step is a stream of the state: the sequential kernel
        chunked = chunk_ok && (dims->seqlen > 1 || !seq_ok);
    if (chunked ? !chunk_ok : !seq_ok)
        return chunked && dims->dtype != SSD_DTYPE_BF16 ? SSD_ERR_UNSUPPORTED_DTYPE : SSD_ERR_UNSUPPORTED;
    if (!chunked)
        return trap_launch(ta, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    if (!pool)
        return SSD_ERR_CUDA;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, chunk_workspace_bytes(ca), pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    ssd_status_t rs = chunk_launch(ca, ws, st);
    if (cudaFreeAsync(ws, st) != cudaSuccess && rs == SSD_OK)
        rs = SSD_ERR_CUDA;
    if (rs == SSD_OK && trap_carry_launch(ta, st) != cudaSuccess)
        rs = SSD_ERR_CUDA;
    return rs;
}

ssd_status_t ssd_conv1d_silu_fwd(const void *xbc, const float *weight, const float *bias,
                                 const void *conv_state, void *x, void *B, void *C, void *conv_state_out,
                                 int32_t kernel_size, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_conv1d_silu_fwd");
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    if (dims->flags != 0 || kernel_size < 1)
        return SSD_ERR_INVALID_DIMS;
    const int64_t es = dims->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const int64_t Cc = (int64_t)dims->nheads * dims->headdim + 2 * (int64_t)dims->ngroups * dims->dstate;
    int64_t xbcb, stb;
    if (!mul_ok(dims->batch * dims->seqlen, Cc * es, &xbcb) || !mul_ok(dims->batch * (kernel_size - 1), Cc * es, &stb))
        return SSD_ERR_INVALID_DIMS;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!xbc || !weight || !x || !B || !C))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {xbc, weight, bias, conv_state, x, B, C, conv_state_out};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    const void *ins[] = {xbc, weight, bias, conv_state};
    const int64_t inb[] = {xbcb, Cc * kernel_size * 4, Cc * 4, stb};
    const void *outs[] = {work ? x : nullptr, work ? B : nullptr, work ? C : nullptr, conv_state_out};
    const int64_t outb[] = {sz.x, sz.bc, sz.bc, stb};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 4; ++i)
            if (overlaps(outs[o], outb[o], ins[i], inb[i]))
                return SSD_ERR_ALIASING;
        for (int o2 = o + 1; o2 < 4; ++o2)
            if (overlaps(outs[o], outb[o], outs[o2], outb[o2]))
                return SSD_ERR_ALIASING;
    }
    NeighborArgs na;
    na.xbc = xbc;
    na.w = weight;
    na.bias = bias;
    na.state_in = conv_state;
    na.x = x;
    na.B = B;
    na.C = C;
    na.state_out = conv_state_out;
    na.kernel_size = kernel_size;
    na.batch = dims->batch;
    na.seqlen = dims->seqlen;
    na.nheads = dims->nheads;
    na.headdim = dims->headdim;
    na.dstate = dims->dstate;
    na.ngroups = dims->ngroups;
    na.dtype = dims->dtype;
    if (!conv_supported(na))
        return SSD_ERR_UNSUPPORTED;
    if (dims->batch == 0)
        return SSD_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->seqlen == 0) {   // no steps: the conv state passes through (zero when not given)
        if (!conv_state_out || stb == 0)
            return SSD_OK;
        const cudaError_t e = conv_state ? cudaMemcpyAsync(conv_state_out, conv_state, (size_t)stb,
                                                           cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(conv_state_out, 0, (size_t)stb, st);
        return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    return conv_launch(na, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_conv_scan_fwd(const void *xbc, const float *conv_weight, const float *conv_bias,
                               const void *conv_state, int32_t kernel_size, const float *dt_raw,
                               const float *dt_bias, const float *A_log, const float *D,
                               const float *init_state, void *y, float *final_state, void *conv_state_out,
                               const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_conv_scan_fwd");
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    if ((dims->flags & ~(SSD_PATH_MASK | SSD_SCHEDULE_REQUEST_MASK)) != 0 || kernel_size < 2 || kernel_size > 4)
        return SSD_ERR_INVALID_DIMS;
    const uint32_t path = dims->flags & SSD_PATH_MASK;
    if (path != SSD_PATH_AUTO && path != SSD_PATH_CHUNKED)
        return SSD_ERR_UNSUPPORTED;
    if (dims->dtype != SSD_DTYPE_BF16)
        return SSD_ERR_UNSUPPORTED_DTYPE;
    const int64_t HP = (int64_t)dims->nheads * dims->headdim, GN = (int64_t)dims->ngroups * dims->dstate;
    const int64_t Cc = HP + 2 * GN;
    if (HP % 8 != 0 || GN % 8 != 0)
        return SSD_ERR_UNSUPPORTED;
    int64_t xbcb, stb;
    if (!mul_ok(dims->batch * dims->seqlen, Cc * 2, &xbcb) || !mul_ok(dims->batch * (kernel_size - 1), Cc * 2, &stb))
        return SSD_ERR_INVALID_DIMS;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!xbc || !conv_weight || !dt_raw || !dt_bias || !A_log || !D || !y))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {xbc, conv_weight, conv_bias, conv_state, dt_raw, dt_bias, A_log, D,
                          init_state, y, final_state, conv_state_out};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    // outputs overlap no input (the scan state may be updated in place) and not each other
    const void *ins[] = {xbc, conv_weight, conv_bias, conv_state, dt_raw, dt_bias, A_log, D, init_state};
    const int64_t inb[] = {xbcb, Cc * kernel_size * 4, Cc * 4, stb, sz.dt, sz.par, sz.par, sz.par, sz.state};
    const void *outs[] = {work ? y : nullptr, final_state, conv_state_out};
    const int64_t outb[] = {sz.x, sz.state, stb};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 9; ++i)
            if (overlaps(outs[o], outb[o], ins[i], inb[i]) && !(o == 1 && i == 8 && outs[o] == ins[i]))
                return SSD_ERR_ALIASING;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlaps(outs[o], outb[o], outs[o2], outb[o2]))
                return SSD_ERR_ALIASING;
    }
    ScanArgs a = make_args(nullptr, dt_raw, dt_bias, A_log, nullptr, nullptr, D, init_state, y, final_state, dims);
    a.conv = true;
    a.xbc = xbc;
    a.conv_w = conv_weight;
    a.conv_b = conv_bias;
    a.conv_state = conv_state;
    a.conv_k = kernel_size;
    a.conv_cc = (int)Cc;
    if (!chunk_supported(a))
        return SSD_ERR_UNSUPPORTED;
    if (dims->batch == 0)
        return SSD_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->seqlen == 0) {   // no steps: both states pass through (zero when not given)
        const void *src[] = {init_state, conv_state};
        void *dst[] = {final_state, conv_state_out};
        const int64_t nb[] = {sz.state, stb};
        for (int i = 0; i < 2; ++i) {
            if (!dst[i] || nb[i] == 0 || src[i] == dst[i])
                continue;
            const cudaError_t e = src[i] ? cudaMemcpyAsync(dst[i], src[i], (size_t)nb[i], cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(dst[i], 0, (size_t)nb[i], st);
            if (e != cudaSuccess)
                return SSD_ERR_CUDA;
        }
        return SSD_OK;
    }
    if (!device_is_gb300_class())
        return SSD_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    if (!pool)
        return SSD_ERR_CUDA;
    // scratch: the convolved B and C, then the chunked path's own
    const size_t bc_bytes = ((size_t)sz.bc + 255) & ~(size_t)255;
    const size_t ws_bytes = chunk_workspace_bytes(a);
    char *buf = nullptr;
    if (cudaMallocFromPoolAsync((void **)&buf, 2 * bc_bytes + ws_bytes, pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    NeighborArgs na;
    na.xbc = xbc;
    na.w = conv_weight;
    na.bias = conv_bias;
    na.state_in = conv_state;
    na.B = buf;
    na.C = buf + bc_bytes;
    na.state_out = conv_state_out;
    na.kernel_size = kernel_size;
    na.batch = dims->batch;
    na.seqlen = dims->seqlen;
    na.nheads = dims->nheads;
    na.headdim = dims->headdim;
    na.dstate = dims->dstate;
    na.ngroups = dims->ngroups;
    na.dtype = dims->dtype;
    ssd_status_t rs = conv_bc_launch(na, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (rs == SSD_OK) {
        a.B = na.B;
        a.C = na.C;
        rs = chunk_launch(a, buf + 2 * bc_bytes, st);
    }
    if (cudaFreeAsync(buf, st) != cudaSuccess && rs == SSD_OK)
        rs = SSD_ERR_CUDA;
    return rs;
}

ssd_status_t ssd_gated_rmsnorm_fwd(const void *y, const void *z, const float *weight, float eps, void *out,
                                   const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_gated_rmsnorm_fwd");
    Sizes sz;
    ssd_status_t s = check_dims(dims, &sz);
    if (s != SSD_OK)
        return s;
    if (dims->flags != 0 || !(eps >= 0.f))
        return SSD_ERR_INVALID_DIMS;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!y || !z || !weight || !out))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {y, z, weight, out};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    if (work && (overlaps(out, sz.x, y, sz.x) || overlaps(out, sz.x, z, sz.x) ||
                 overlaps(out, sz.x, weight, (int64_t)dims->nheads * dims->headdim * 4)))
        return SSD_ERR_ALIASING;
    NeighborArgs na;
    na.y = y;
    na.z = z;
    na.w = weight;
    na.out = out;
    na.eps = eps;
    na.batch = dims->batch;
    na.seqlen = dims->seqlen;
    na.nheads = dims->nheads;
    na.headdim = dims->headdim;
    na.dtype = dims->dtype;
    if (!gnorm_supported(na))
        return SSD_ERR_UNSUPPORTED;
    if (!work)
        return SSD_OK;
    return gnorm_launch(na, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_scan_bwd(const void *x, const float *dt_raw, const float *dt_bias, const float *A_log,
                          const void *B, const void *C, const float *D, const float *init_state, const void *dy,
                          const float *d_final, float *dx, float *ddt_raw, float *ddt_bias, float *dA_log,
                          float *dB, float *dC, float *dD, float *d_init, const ssd_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_scan_bwd");
    Sizes sz;
    if (!dims)
        return SSD_ERR_NULL_PTR;
    ssd_dims_t dchk = *dims;   // (the backward's own flags are checked here, the rest by check_dims)
    dchk.flags &= ~(SSD_BWD_FP32_FORM | SSD_BWD_SPLIT_STATES);
    ssd_status_t s = check_dims(&dchk, &sz);
    if (s != SSD_OK)
        return s;
    if ((dims->flags & ~(SSD_PATH_MASK | SSD_BWD_FP32_FORM | SSD_BWD_SPLIT_STATES)) != 0)
        return SSD_ERR_INVALID_DIMS;
    const uint32_t path = dims->flags & SSD_PATH_MASK;
    if (path != SSD_PATH_AUTO && path != SSD_PATH_SEQUENTIAL && path != SSD_PATH_CHUNKED)
        return SSD_ERR_UNSUPPORTED;
    const bool work = dims->batch > 0 && dims->seqlen > 0;
    if (work && (!x || !dt_raw || !dt_bias || !A_log || !B || !C || !D || !dy || !dx || !ddt_raw || !ddt_bias ||
                 !dA_log || !dB || !dC || !dD))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {x, dt_raw, dt_bias, A_log, B, C, D, init_state, dy, d_final,
                          dx, ddt_raw, ddt_bias, dA_log, dB, dC, dD, d_init};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr))
            return SSD_ERR_MISALIGNED;
    // fp32 gradients: dx [B,L,H,P], ddt_raw [B,L,H], dB/dC [B,L,G,N], per-head [H], d_init [B,H,P,N]
    const int64_t es = dims->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const int64_t x32 = sz.x / es * 4, bc32 = sz.bc / es * 4;
    const void *ins[] = {x, dt_raw, dt_bias, A_log, B, C, D, init_state, dy, d_final};
    const int64_t inb[] = {sz.x, sz.dt, sz.par, sz.par, sz.bc, sz.bc, sz.par, sz.state, sz.x, sz.state};
    const void *outs[] = {dx, ddt_raw, ddt_bias, dA_log, dB, dC, dD, d_init};
    const int64_t outb[] = {x32, sz.dt, sz.par, sz.par, bc32, bc32, sz.par, sz.state};
    if (work)
        for (int o = 0; o < 8; ++o) {
            for (int i = 0; i < 10; ++i)
                if (overlaps(outs[o], outb[o], ins[i], inb[i]))
                    return SSD_ERR_ALIASING;
            for (int o2 = o + 1; o2 < 8; ++o2)
                if (overlaps(outs[o], outb[o], outs[o2], outb[o2]))
                    return SSD_ERR_ALIASING;
        }
    BwdArgs ba;
    ba.x = x;
    ba.B = B;
    ba.C = C;
    ba.dy = dy;
    ba.dt_raw = dt_raw;
    ba.dt_bias = dt_bias;
    ba.A_log = A_log;
    ba.D = D;
    ba.init_state = init_state;
    ba.d_final = d_final;
    ba.dx = dx;
    ba.ddt_raw = ddt_raw;
    ba.ddt_bias = ddt_bias;
    ba.dA_log = dA_log;
    ba.dB = dB;
    ba.dC = dC;
    ba.dD = dD;
    ba.d_init = d_init;
    ba.batch = dims->batch;
    ba.seqlen = dims->seqlen;
    ba.nheads = dims->nheads;
    ba.headdim = dims->headdim;
    ba.dstate = dims->dstate;
    ba.ngroups = dims->ngroups;
    ba.dtype = dims->dtype;
    ba.path = path;
    ba.fp32_form = (dims->flags & SSD_BWD_FP32_FORM) != 0;
    ba.split_states = (dims->flags & SSD_BWD_SPLIT_STATES) != 0;
    if (path == SSD_PATH_AUTO)
        ba.path = bwd_chunk_supported(ba) ? SSD_PATH_CHUNKED : SSD_PATH_SEQUENTIAL;
    if (!bwd_supported(ba))
        return SSD_ERR_UNSUPPORTED;
    if (!work)
        return SSD_OK;   // (empty work: nothing is written)
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return SSD_ERR_CUDA;
    cudaMemPool_t pool = scratch_pool(dev);
    if (!pool)
        return SSD_ERR_CUDA;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, bwd_workspace_bytes(ba), pool, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    ssd_status_t rs = bwd_launch(ba, ws, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (cudaFreeAsync(ws, st) != cudaSuccess && rs == SSD_OK)
        rs = SSD_ERR_CUDA;
    return rs;
}

ssd_status_t ssd_paged_plan(const int32_t *lens, const int32_t *new_lens, int32_t *block_table, int32_t *free_ring,
                            const int64_t *ring_pos, int32_t *lens_out, int32_t *granted, int32_t *start,
                            int32_t *positions, int32_t *token_req, int64_t *slots, int64_t *ring_pos_out,
                            int32_t *counts, const ssd_plan_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_paged_plan");
    if (!dims)
        return SSD_ERR_NULL_PTR;
    const int64_t lim = INT64_C(1) << 31;
    if (dims->flags != 0 || dims->reserved != 0 || dims->nreq < 0 || dims->max_tokens < 0 || dims->max_tokens >= lim ||
        dims->ring_size < 1 || dims->ring_size >= lim || dims->page_size < 1 || dims->max_pages < 1 ||
        (int64_t)dims->page_size * dims->max_pages >= lim)
        return SSD_ERR_INVALID_DIMS;
    if (dims->nreq > SSD_PLAN_MAX_REQUESTS)
        return SSD_ERR_UNSUPPORTED;
    const int64_t n = dims->nreq, T = dims->max_tokens;
    if (!free_ring || !ring_pos || !start || !ring_pos_out || !counts ||
        (n > 0 && (!lens || !new_lens || !block_table || !lens_out || !granted)) ||
        (T > 0 && (!positions || !token_req || !slots)))
        return SSD_ERR_NULL_PTR;
    struct { const void *p; int64_t bytes; bool out; } a[] = {
        {lens, n * 4, false}, {new_lens, n * 4, false}, {ring_pos, 16, false},
        {block_table, n * dims->max_pages * 4, true}, {free_ring, dims->ring_size * 4, true}, {lens_out, n * 4, true},
        {granted, n * 4, true}, {start, (n + 1) * 4, true}, {positions, T * 4, true}, {token_req, T * 4, true},
        {slots, T * 8, true}, {ring_pos_out, 16, true}, {counts, 16, true}};
    constexpr int na = sizeof(a) / sizeof(a[0]);
    for (const auto &x : a)
        if (!aligned16(x.p))
            return SSD_ERR_MISALIGNED;
    for (int i = 0; i < na; ++i)
        for (int j = i + 1; j < na; ++j) {
            const bool in_place = a[i].p == a[j].p && ((a[i].p == lens && a[j].p == lens_out && i == 0 && j == 5) ||
                                                       (i == 2 && j == 11));
            if ((a[i].out || a[j].out) && !in_place && overlaps(a[i].p, a[i].bytes, a[j].p, a[j].bytes))
                return SSD_ERR_ALIASING;
        }
    PlanArgs pa;
    pa.lens = lens;
    pa.new_lens = new_lens;
    pa.table = block_table;
    pa.ring = free_ring;
    pa.ring_pos = ring_pos;
    pa.lens_out = lens_out;
    pa.granted = granted;
    pa.start = start;
    pa.positions = positions;
    pa.token_req = token_req;
    pa.slots = slots;
    pa.ring_pos_out = ring_pos_out;
    pa.counts = counts;
    pa.nreq = (int)n;
    pa.max_tokens = (int)T;
    pa.ring_size = (int)dims->ring_size;
    pa.page_size = dims->page_size;
    pa.max_pages = dims->max_pages;
    return plan_launch(pa, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_qk_norm_rope_fwd(const void *q, const void *k, const void *v, const float *q_weight,
                                  const float *k_weight, const float *cos, const float *sin, const int32_t *positions,
                                  void *q_out, void *k_out, void *k_cache, void *v_cache, const int64_t *slots,
                                  const ssd_qk_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_qk_norm_rope_fwd");
    const bool cache = k_cache || v_cache || slots;
    const ssd_status_t s = check_qk_dims(dims, cache, false);
    if (s != SSD_OK)
        return s;
    const int64_t T = dims->ntokens, D = dims->headdim, es = (int64_t)elem_size(dims->dtype);
    if (T > 0 && (!q || !k || !positions || !q_out || (!k_out && !cache) ||
                  (dims->rotary_dim > 0 && dims->max_pos > 0 && (!cos || !sin))))
        return SSD_ERR_NULL_PTR;
    if (cache && (!k_cache || !v_cache || (T > 0 && (!v || !slots))))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {q, k, v, q_weight, k_weight, cos, sin, q_out, k_out, k_cache, v_cache};
    for (const void *p : ptrs)
        if (!aligned16(p))
            return SSD_ERR_MISALIGNED;
    if (!aligned(positions, 4) || !aligned(slots, 8))
        return SSD_ERR_MISALIGNED;
    const int64_t Hq = dims->nheads_q, Hk = dims->nheads_k, w = D * es;
    const int64_t tab = dims->max_pos * (dims->rotary_dim / 2) * 4;
    const Strided vq = view(q, T, Hq, dims->q_stride, w, es), vk = view(k, T, Hk, dims->k_stride, w, es);
    const Strided vv = view(cache ? v : nullptr, T, Hk, dims->v_stride, w, es);
    const Strided oq = view(q_out, T, Hq, dims->qo_stride, w, es), ok = view(k_out, T, Hk, dims->ko_stride, w, es);
    const Strided *ins[] = {&vq, &vk, &vv}, *outs[] = {&oq, &ok};
    const struct { const void *p; int64_t bytes; } flat[] = {{q_weight, D * 4}, {k_weight, D * 4}, {cos, tab}, {sin, tab},
                                                              {positions, T * 4}, {slots, cache ? T * 8 : 0}};
    const int64_t kcb = cache ? cache_extent(dims->npages, dims->page_size, Hk, dims->kc_stride, D, es) : 0;
    const int64_t vcb = cache ? cache_extent(dims->npages, dims->page_size, Hk, dims->vc_stride, D, es) : 0;
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 3; ++i)
            if (overlaps(*outs[o], *ins[i]) && !(o == i && same_view(*outs[o], *ins[i])))
                return SSD_ERR_ALIASING;
        for (const auto &f : flat)
            if (overlaps(outs[o]->p, outs[o]->extent(), f.p, f.bytes))
                return SSD_ERR_ALIASING;
        if (overlaps(outs[o]->p, outs[o]->extent(), k_cache, kcb) || overlaps(outs[o]->p, outs[o]->extent(), v_cache, vcb))
            return SSD_ERR_ALIASING;
    }
    if (overlaps(oq, ok) || !distinct_rows(oq) || !distinct_rows(ok))
        return SSD_ERR_ALIASING;
    for (int i = 0; i < 3; ++i)
        if (overlaps(ins[i]->p, ins[i]->extent(), k_cache, kcb) || overlaps(ins[i]->p, ins[i]->extent(), v_cache, vcb))
            return SSD_ERR_ALIASING;
    for (const auto &f : flat)
        if (overlaps(f.p, f.bytes, k_cache, kcb) || overlaps(f.p, f.bytes, v_cache, vcb))
            return SSD_ERR_ALIASING;
    if (cache) {
        const auto rows = [&](const void *p, const int64_t *s) {
            return Rows{p, w, {dims->npages, dims->page_size, Hk}, {s[0] * es, s[1] * es, s[2] * es}};
        };
        const Rows kr = rows(k_cache, dims->kc_stride), vr = rows(v_cache, dims->vc_stride);
        if (overlaps(kr, vr) || !distinct_rows(kr) || !distinct_rows(vr))
            return SSD_ERR_ALIASING;
    }
    if (T == 0)
        return SSD_OK;
    QkArgs qa{};
    qa.q = q;
    qa.k = k;
    qa.v = v;
    qa.qw = q_weight;
    qa.kw = k_weight;
    qa.cos = cos;
    qa.sin = sin;
    qa.positions = positions;
    qa.qo = q_out;
    qa.ko = k_out;
    qa.kc = k_cache;
    qa.vc = v_cache;
    qa.slots = slots;
    qa.d = *dims;
    return qk_fwd_launch(qa, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_qk_norm_rope_bwd_workspace_size(const ssd_qk_dims_t *dims, uint64_t *bytes)
{
    if (!bytes)
        return SSD_ERR_NULL_PTR;
    const ssd_status_t s = check_qk_dims(dims, false, true);
    if (s != SSD_OK)
        return s;
    *bytes = qk_bwd_workspace_bytes(*dims);
    return SSD_OK;
}

ssd_status_t ssd_qk_norm_rope_bwd(const void *q, const void *k, const float *q_weight, const float *k_weight,
                                  const float *cos, const float *sin, const int32_t *positions, const void *dq_out,
                                  const void *dk_out, void *dq, void *dk, float *dq_weight, float *dk_weight,
                                  void *workspace, uint64_t workspace_bytes, const ssd_qk_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_qk_norm_rope_bwd");
    const ssd_status_t s = check_qk_dims(dims, false, true);
    if (s != SSD_OK)
        return s;
    const int64_t T = dims->ntokens, D = dims->headdim, es = (int64_t)elem_size(dims->dtype);
    if (T > 0 && (!q || !k || !positions || !dq_out || !dk_out || !dq || !dk ||
                  (dims->rotary_dim > 0 && dims->max_pos > 0 && (!cos || !sin))))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {q, k, q_weight, k_weight, cos, sin, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p))
            return SSD_ERR_MISALIGNED;
    if (!aligned(positions, 4))
        return SSD_ERR_MISALIGNED;
    const int64_t Hq = dims->nheads_q, Hk = dims->nheads_k, w = D * es;
    const int64_t tab = dims->max_pos * (dims->rotary_dim / 2) * 4;
    const Strided v[] = {view(q, T, Hq, dims->q_stride, w, es), view(k, T, Hk, dims->k_stride, w, es),
                         view(dq_out, T, Hq, dims->qo_stride, w, es), view(dk_out, T, Hk, dims->ko_stride, w, es)};
    const Strided o[] = {view(dq, T, Hq, dims->dq_stride, w, es), view(dk, T, Hk, dims->dk_stride, w, es)};
    const int64_t wsb = workspace ? (int64_t)(workspace_bytes > (uint64_t)INT64_MAX ? INT64_MAX : workspace_bytes) : 0;
    // every other array as a flat range, outputs last
    const struct { const void *p; int64_t bytes; } flat[] = {{q_weight, D * 4}, {k_weight, D * 4}, {cos, tab}, {sin, tab},
                                                              {positions, T * 4}, {dq_weight, D * 4}, {dk_weight, D * 4},
                                                              {workspace, wsb}};
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlaps(o[i], v[j]) && !(j == i + 2 && same_view(o[i], v[j])))
                return SSD_ERR_ALIASING;
        for (const auto &f : flat)
            if (overlaps(o[i].p, o[i].extent(), f.p, f.bytes))
                return SSD_ERR_ALIASING;
    }
    if (overlaps(o[0], o[1]) || !distinct_rows(o[0]) || !distinct_rows(o[1]))
        return SSD_ERR_ALIASING;
    for (int i = 5; i < 8; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlaps(v[j].p, v[j].extent(), flat[i].p, flat[i].bytes))
                return SSD_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (overlaps(flat[j].p, flat[j].bytes, flat[i].p, flat[i].bytes))
                return SSD_ERR_ALIASING;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: the weights' gradients are zero
        if ((dq_weight && cudaMemsetAsync(dq_weight, 0, (size_t)D * 4, st) != cudaSuccess) ||
            (dk_weight && cudaMemsetAsync(dk_weight, 0, (size_t)D * 4, st) != cudaSuccess))
            return SSD_ERR_CUDA;
        return SSD_OK;
    }
    QkArgs qa{};
    qa.q = q;
    qa.k = k;
    qa.qw = q_weight;
    qa.kw = k_weight;
    qa.cos = cos;
    qa.sin = sin;
    qa.positions = positions;
    qa.qo = const_cast<void *>(dq_out);
    qa.ko = const_cast<void *>(dk_out);
    qa.dq = dq;
    qa.dk = dk;
    qa.dqw = dq_weight;
    qa.dkw = dk_weight;
    qa.d = *dims;
    const size_t need = dq_weight || dk_weight ? qk_bwd_workspace_bytes(*dims) : 0;
    return with_workspace(workspace, workspace_bytes, need, st, [&](void *ws) { return qk_bwd_launch(qa, ws, st); });
}

ssd_status_t ssd_paged_attn_workspace_size(const ssd_attn_dims_t *dims, uint64_t *bytes)
{
    if (!bytes)
        return SSD_ERR_NULL_PTR;
    const ssd_status_t s = check_attn_dims(dims);
    if (s != SSD_OK)
        return s;
    *bytes = dims->nrows > 0 ? attn_workspace_bytes(*dims) : 0;
    return SSD_OK;
}

ssd_status_t ssd_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                                const int32_t *positions, const int32_t *start, void *out, float *lse, void *workspace,
                                uint64_t workspace_bytes, const ssd_attn_dims_t *dims, void *stream)
{
    SSD_NVTX_RANGE("ssd_paged_attn_fwd");
    const ssd_status_t s = check_attn_dims(dims);
    if (s != SSD_OK)
        return s;
    if (!start && dims->nrows != dims->nreq)
        return SSD_ERR_INVALID_DIMS;
    if (start && dims->nreq > SSD_ATTN_MAX_REQUESTS)
        return SSD_ERR_UNSUPPORTED;
    const int64_t R = dims->nrows, D = dims->headdim, es = (int64_t)elem_size(dims->dtype);
    if (R > 0 && (!q || !positions || !out || (dims->nreq > 0 && !block_table) ||
                  (dims->npages > 0 && (!k_cache || !v_cache))))
        return SSD_ERR_NULL_PTR;
    const void *ptrs[] = {q, k_cache, v_cache, out, lse, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p))
            return SSD_ERR_MISALIGNED;
    if (!aligned(block_table, 4) || !aligned(positions, 4) || !aligned(start, 4))
        return SSD_ERR_MISALIGNED;
    const int64_t w = D * es;
    const Strided vq = view(q, R, dims->nheads, dims->q_stride, w, es), vo = view(out, R, dims->nheads, dims->o_stride, w, es);
    if ((overlaps(vo, vq) && !same_view(vo, vq)) || !distinct_rows(vo))
        return SSD_ERR_ALIASING;
    const int64_t wsb = workspace ? (int64_t)(workspace_bytes > (uint64_t)INT64_MAX ? INT64_MAX : workspace_bytes) : 0;
    const struct { const void *p; int64_t bytes; } in[] = {
        {k_cache, cache_extent(dims->npages, dims->page_size, dims->nkv, dims->kc_stride, D, es)},
        {v_cache, cache_extent(dims->npages, dims->page_size, dims->nkv, dims->vc_stride, D, es)},
        {block_table, dims->nreq > 0 ? ((dims->nreq - 1) * dims->table_stride + dims->max_pages) * 4 : 0},
        {positions, R * 4}, {start, (dims->nreq + 1) * 4}, {q, vq.extent()}};
    const struct { const void *p; int64_t bytes; } ob[] = {{out, vo.extent()}, {lse, R * dims->nheads * 4}, {workspace, wsb}};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < (o == 0 ? 5 : 6); ++i)
            if (overlaps(ob[o].p, ob[o].bytes, in[i].p, in[i].bytes))
                return SSD_ERR_ALIASING;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlaps(ob[o].p, ob[o].bytes, ob[o2].p, ob[o2].bytes))
                return SSD_ERR_ALIASING;
    }
    if (R == 0)
        return SSD_OK;
    AttnArgs aa;
    aa.q = q;
    aa.kc = k_cache;
    aa.vc = v_cache;
    aa.table = block_table;
    aa.positions = positions;
    aa.start = start;
    aa.out = out;
    aa.lse = lse;
    aa.d = *dims;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_workspace(workspace, workspace_bytes, attn_workspace_bytes(*dims), st,
                          [&](void *ws) { return attn_launch(aa, ws, st); });
}

}  // extern "C"
