/*
 * libssd -- forward Mamba-2 SSD (structured state-space duality) scan on one
 * NVIDIA GB300 (sm_103a).  Plain C ABI: host or device pointers, sizes and a
 * CUDA stream handle; no framework types.
 *
 * The operation (per batch row b and head h, for t = 0 .. L-1):
 *
 *   dt_t  = softplus(dt_raw[b,t,h] + dt_bias[h])
 *   A_h   = -exp(A_log[h])                        A_log stores log(-A)
 *   h_t   = exp(dt_t * A_h) * h_{t-1} + dt_t * B[b,t,g] x[b,t,h]^T      (N x P)
 *   y[b,t,h] = C[b,t,g]^T h_t + D[h] * x[b,t,h]
 *
 * with g = h * G / H (contiguous blocks of H/G heads share a group) and h_{-1}
 * the initial state (zero when none is given).  Defined by the SSD module of
 * @seanhogg/builderforce-memory-engine 2026.6.18 (package/dist/kernels/
 * ssd.js and ssd.d.ts, module header: scalar decay per head, MIMO state per
 * head, chunked evaluation with a carried state, buffer layouts), taken with
 * A = -exp(A_log), input term dt * B x^T and a readout per channel p.  The
 * chunked evaluation (chunks of Q steps, chunk states passed from chunk to
 * chunk) follows the chunked-scan structure of mamba-rs 0.2.1
 * src/mamba3_siso/gpu/mamba3_gpu.rs (parallel branch of the forward layer:
 * decay cumsum, chunk state, state passing, chunk scan) applied to the
 * Mamba-2 recurrence above.
 *
 * Layouts: row-major and contiguous.
 *   x, y                   [B, L, H, P]   dtype (bf16 or fp32)
 *   dt_raw                 [B, L, H]      fp32
 *   B, C                   [B, L, G, N]   dtype
 *   dt_bias, A_log, D      [H]            fp32
 *   init_state, final_state [B, H, P, N]  fp32 (state stored P-major, N-minor)
 */
#ifndef LIBSSD_SSD_H
#define LIBSSD_SSD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_ABI_VERSION 2

typedef enum ssd_dtype {
    SSD_DTYPE_F32 = 0,   /* x, B, C, y are fp32 */
    SSD_DTYPE_BF16 = 1   /* x, B, C, y are bf16; arithmetic accumulates in fp32 */
} ssd_dtype_t;

typedef enum ssd_status {
    SSD_OK = 0,
    SSD_ERR_INVALID_DIMS = 1,   /* a size is negative/zero where it may not be, H % G != 0, overflow */
    SSD_ERR_NULL_PTR = 2,       /* a required pointer is NULL */
    SSD_ERR_MISALIGNED = 3,     /* a pointer is not 16-byte aligned */
    SSD_ERR_UNSUPPORTED = 4,    /* shape or requested path not supported */
    SSD_ERR_CUDA = 5,           /* a CUDA runtime/driver call failed; nothing further enqueued */
    SSD_ERR_TIMEOUT = 6,        /* a kernel gave up a bounded wait (read via ssd_get_device_error) */
    SSD_ERR_ALIASING = 7,       /* y overlaps an input, or the two states overlap partially */
    SSD_ERR_SCRATCH_LIMIT = 8,  /* the scratch needed exceeds the buffer the call may use (the fixed
                                   array of ssd_scan_fwd_noalloc, the workspace of ssd_scan_fwd_ws) */
    SSD_ERR_UNSUPPORTED_DTYPE = 9   /* dims->dtype is not an ssd_dtype_t, or the path requested (or,
                                       for ssd_scan_fwd_noalloc, the only path it has) does not take it:
                                       the chunked tcgen05 path takes bf16 only */
} ssd_status_t;

/* Kernel path selection, in ssd_dims_t.flags (low 4 bits). */
#define SSD_PATH_AUTO 0u        /* decode step for seqlen 1, else the chunked tensor-core path where
                                   supported, else sequential */
#define SSD_PATH_SEQUENTIAL 1u  /* direct recurrence, fp32 FFMA (any P, N up to 2048; fp32 or bf16) */
#define SSD_PATH_CHUNKED 2u     /* chunked tcgen05 path: bf16, P = 64, N = 128, Q % 64 == 0, (H/G) even */
#define SSD_PATH_DECODE 3u      /* one step (seqlen 1), fp32 FFMA: any P, N % 4 == 0 and N <= 512; fp32 or
                                   bf16.  SSD_PATH_AUTO takes it whenever seqlen == 1 and it applies */
#define SSD_PATH_MASK 0xFu
/* Diagnostic, in ssd_dims_t.flags: on the chunked path, the first unit of every
 * chain waits for a state handoff that nothing publishes, with the bounded waits
 * shortened to 20 ms.  The launch then records SSD_ERR_TIMEOUT (read with
 * ssd_get_device_error), stops every warp, drains its own copies and MMAs and
 * returns; y and final_state are undefined.  It exercises the failure path
 * without faulting the GPU.  Ignored by the sequential path. */
#define SSD_DIAG_STALL_HANDOFF 0x100u
/* In ssd_dims_t.flags of ssd_scan_bwd only: run the chunk form's fp32
 * contractions even where its tensor-core gradient pass applies (bf16 inputs,
 * P = 64, N = 128).  The tensor-core pass rounds the masked decay products
 * and the chunk states to bf16 operands; the fp32 form does not. */
#define SSD_BWD_FP32_FORM 0x200u
/* In ssd_dims_t.flags of ssd_scan_bwd only: where the tensor-core form applies,
 * compute the chunk states and link them in two launches (every chunk at once,
 * then the chains) rather than in one launch that walks each (b, h) through its
 * chunks with the running state in TMEM.  The library takes the one-launch walk
 * when 2 B H fills the GPU's SMs or the sequence has at most 8 chunks of 64
 * steps.  Both give the same chunk states up to the order of fp32 additions. */
#define SSD_BWD_SPLIT_STATES 0x400u

/* Schedules of the chunked path (see ssd_chunk_schedule).  One may be requested
 * in ssd_dims_t.flags as (SSD_SCHEDULE_x << SSD_SCHEDULE_SHIFT); 0 there lets
 * the library choose.  A split request for a sequence of a single chunk runs
 * the range schedule (there is nothing to split).  Ignored by the sequential
 * path. */
#define SSD_SCHEDULE_NONE 0
#define SSD_SCHEDULE_RANGES 1
#define SSD_SCHEDULE_PIECES 2
#define SSD_SCHEDULE_SPLIT 3
#define SSD_SCHEDULE_SHIFT 4
#define SSD_SCHEDULE_REQUEST_MASK 0x30u

typedef struct ssd_dims {
    int64_t batch;     /* B >= 0 */
    int64_t seqlen;    /* L >= 0; need not be a multiple of chunk (ragged last chunk) */
    int32_t nheads;    /* H >= 1 */
    int32_t headdim;   /* P >= 1 */
    int32_t dstate;    /* N >= 1 */
    int32_t ngroups;   /* G >= 1, H % G == 0 */
    int32_t chunk;     /* Q >= 1: chunk length of the chunked evaluation (ignored by the sequential path) */
    int32_t dtype;     /* ssd_dtype_t of x, B, C and y */
    uint32_t flags;    /* SSD_PATH_* | optional schedule request | optional SSD_DIAG_STALL_HANDOFF */
    uint32_t reserved; /* must be 0 */
} ssd_dims_t;

/*
 * ssd_scan_fwd -- the forward scan on device memory.
 *
 * All array arguments are DEVICE pointers of the current device, owned by the
 * caller, contiguous in the layouts above and 16-byte aligned.  init_state may
 * be NULL (zero initial state); final_state may be NULL (not returned).
 * init_state and final_state may be the same pointer (in-place state update)
 * but must not overlap otherwise; y must not overlap any input.
 * `stream` is a cudaStream_t (NULL = legacy default stream).  The call only
 * enqueues work on `stream`: it never synchronises, and returns before the
 * results are ready.  Scratch memory (chunk-handoff flags, and chunk states
 * when final_state is NULL) is taken stream-ordered from a library-owned
 * memory pool and released stream-ordered after the kernel.
 * Errors: returns a status; on any status other than SSD_OK nothing was
 * enqueued, except SSD_ERR_CUDA raised by a launch itself.  A kernel that
 * exceeds a bounded wait (about 2 s) records SSD_ERR_TIMEOUT in a device
 * error word, stops, and leaves y undefined; read it with
 * ssd_get_device_error.
 */
ssd_status_t ssd_scan_fwd(const void *x, const float *dt_raw, const float *dt_bias,
                          const float *A_log, const void *B, const void *C, const float *D,
                          const float *init_state, void *y, float *final_state,
                          const ssd_dims_t *dims, void *stream);

/*
 * ssd_scan_fwd_host -- the same scan on HOST buffers (end-to-end use).
 *
 * Arguments as ssd_scan_fwd but every array is a host pointer (pinned memory
 * gives asynchronous copies; pageable works).  The call allocates device
 * buffers stream-ordered, copies the inputs in, runs the scan, copies y (and
 * final_state when non-NULL) back, releases the buffers, and synchronises
 * `stream` before returning, so the host outputs are ready on SSD_OK.
 * Calls of 32 MiB or more with several batch rows run in up to 8 pieces of
 * whole rows through three library-owned streams (copies in, scan, copies
 * out), ordered after and joined back into `stream` by events, so that the
 * two copy directions and the scan overlap.  Every piece takes the schedule
 * the whole batch would, and the results are bitwise those of ssd_scan_fwd.
 */
ssd_status_t ssd_scan_fwd_host(const void *x, const float *dt_raw, const float *dt_bias,
                               const float *A_log, const void *B, const void *C,
                               const float *D, const float *init_state, void *y,
                               float *final_state, const ssd_dims_t *dims, void *stream);

/*
 * ssd_scan_fwd_workspace_size -- bytes of scratch that ssd_scan_fwd_ws needs for
 * these dims on the current device, in *bytes (0 when the call needs none:
 * empty work or the sequential path).  The chunked path's scratch holds the
 * chunk-unit handoff flags and, when a chain is split into several units,
 * the handed-over states (the inter-chunk state passing of the chunked
 * evaluation; @seanhogg/builderforce-memory-engine, dist/kernels/ssd.js, module
 * header: chunked evaluation with a carried state).  The schedule, and so the
 * size, depends on the device's SM count.  Host only; launches nothing.
 * Returns SSD_OK, or an error for invalid or unsupported dims (as
 * ssd_select_path), or SSD_ERR_NULL_PTR.
 */
ssd_status_t ssd_scan_fwd_workspace_size(const ssd_dims_t *dims, uint64_t *bytes);

/*
 * ssd_scan_fwd_ws -- ssd_scan_fwd with caller-provided scratch.
 *
 * Arguments as ssd_scan_fwd, plus `workspace`: a DEVICE buffer of
 * `workspace_bytes` bytes, owned by the caller, 16-byte aligned, overlapping
 * no other argument.  It must hold ssd_scan_fwd_workspace_size(dims) bytes
 * (it may be NULL when that is 0); its contents on entry do not matter and
 * are undefined afterwards.  The call allocates nothing.  Two calls whose
 * kernels may overlap in time must not share a workspace.
 * Errors as ssd_scan_fwd, plus SSD_ERR_SCRATCH_LIMIT when workspace_bytes is
 * smaller than needed (nothing enqueued); a misaligned or overlapping
 * workspace gives SSD_ERR_MISALIGNED or SSD_ERR_ALIASING before any CUDA call.
 */
ssd_status_t ssd_scan_fwd_ws(const void *x, const float *dt_raw, const float *dt_bias,
                             const float *A_log, const void *B, const void *C, const float *D,
                             const float *init_state, void *y, float *final_state,
                             void *workspace, uint64_t workspace_bytes, const ssd_dims_t *dims,
                             void *stream);

/*
 * ssd_scan_fwd_noalloc -- ssd_scan_fwd on the chunked path without any
 * device-memory allocation.
 *
 * No counterpart in the paper: an engineering variant for callers that cannot
 * let a library allocate device memory during a call (a process that reserves
 * the device up front in an arena of its own, or a driver or virtualised
 * device without stream-ordered memory pools).
 *
 * Arguments, layouts and ownership as ssd_scan_fwd.  Runs the same chunked
 * tcgen05 kernel with its scratch in a fixed 32 MiB array that the library
 * module holds per device.  The array's device address is looked up on the
 * first call on a device, with that device current, and again after the
 * device's context has changed (cudaDeviceReset); make that first call before
 * any stream capture.  The call calls no allocator.
 * Errors as ssd_scan_fwd, plus:
 *   SSD_ERR_UNSUPPORTED    the chunked path does not support these dims, or
 *                          dims->flags requests a path other than
 *                          SSD_PATH_AUTO or SSD_PATH_CHUNKED (the sequential
 *                          and decode paths need no scratch: call ssd_scan_fwd),
 *                          or requests SSD_SCHEDULE_SPLIT;
 *   SSD_ERR_UNSUPPORTED_DTYPE  dims->dtype is not bf16;
 *   SSD_ERR_SCRATCH_LIMIT  the kernel would need more than 32 MiB of scratch;
 *                          nothing is enqueued.  The call never takes
 *                          SSD_SCHEDULE_SPLIT, and takes SSD_SCHEDULE_PIECES
 *                          (one 64 KiB state slot and 64 B of flags per SM)
 *                          wherever the schedule ssd_scan_fwd would take needs
 *                          more than the array, so only a device of more than
 *                          about 500 SMs gets this error;
 *   SSD_ERR_CUDA           the array's address could not be obtained.
 * Concurrency: the array is shared by all calls on a device.  Calls whose
 * kernels may overlap in time on one device (different streams, or threads
 * without ordering between them) race on it and give wrong results or time
 * out; calls ordered on one stream are safe.
 */
ssd_status_t ssd_scan_fwd_noalloc(const void *x, const float *dt_raw, const float *dt_bias,
                                  const float *A_log, const void *B, const void *C,
                                  const float *D, const float *init_state, void *y,
                                  float *final_state, const ssd_dims_t *dims, void *stream);

/*
 * ssd_trap_scan_fwd -- the trapezoidal (Mamba-3 SISO) scan, forward.
 *
 * The Mamba-3 SISO GPU forward of the pages (mamba-rs 0.2.1,
 * mamba3_siso/gpu/mamba3_gpu.rs) replaces the exponential recurrence by a
 * trapezoidal one in three coefficients and keeps the last step's k and v as
 * extra carried state (module header of its forward pass; step F5b:
 * alpha = exp(a dt), beta = alpha dt (1 - trap), gamma = trap dt).  Per batch row b and head h, with v = x, k = B, q = C of
 * the head's group g = h / (H/G):
 *   h_t = alpha_t h_{t-1} + beta_t k_{t-1} v_{t-1}^T + gamma_t k_t v_t^T
 *   y_t = q_t^T h_t + D_h v_t
 * where k_{-1}, v_{-1} are the carried k_state and v_state.  The pages print
 * the coefficients and the k/v states but not the recurrence; the form above
 * is the reading they support.  The coefficient step is fused: the call takes
 * dt, a and trap per token.
 *
 * Arguments are DEVICE pointers of the current device, owned by the caller,
 * contiguous, 16-byte aligned; dims as for ssd_scan_fwd (dtype: x, B, C, y
 * and the k/v states).  flags: a path and, for the chunked kernel, a schedule
 * request as for ssd_scan_fwd.  SSD_PATH_CHUNKED is the chunked tcgen05 kernel
 * in a trapezoidal mode (same limits and schedules as for ssd_scan_fwd: bf16,
 * P = 64, N = 128, chunk % 64 == 0, (H/G) even; scratch from the library pool;
 * one more small launch writes k_final / v_final).  The mode evaluates the
 * recurrence on the shifted state h~_t = h_t + (beta_{t+1}/alpha_{t+1})
 * k_t v_t^T, which is linear with decay alpha_t, so the split schedule applies
 * unchanged; its first pass starts each chain from h0 + dt_0 (1 - trap_0)
 * k0 v0^T.  SSD_PATH_SEQUENTIAL is a
 * sequential kernel (fp32 arithmetic).  SSD_PATH_AUTO takes the chunked kernel
 * where it applies and seqlen > 1, else the sequential one.
 *   v     [B,L,H,P]   k, q [B,L,G,N]   (dtype)
 *   dt, a, trap [B,L,H] fp32: step size (> 0), per-token decay rate (a <= 0 for
 *                       a decaying state), mixing weight in [0, 1]
 *   D [H] fp32
 *   h0, h_final [B,H,P,N] fp32; k0, k_final [B,H,N] (dtype); v0, v_final
 *                       [B,H,P] (dtype).  Inputs may be NULL (zero), outputs
 *                       NULL (not written).  Each output may be the same
 *                       pointer as its input (in place) but must not
 *                       overlap anything else.  k_final[b,h] = k[b,L-1,g] and
 *                       v_final[b,h] = v[b,L-1,h]: the next call continues
 *                       from (h_final, k_final, v_final).
 *   y [B,L,H,P] (dtype), overlapping no input.
 * The sequential kernel supports N % 4 == 0, N <= 512; P <= 128 for
 * N <= 128, P <= 64 for N <= 256, P <= 32 for N <= 512; fp32 or bf16.
 * Returns SSD_OK, or an error as ssd_scan_fwd (SSD_ERR_INVALID_DIMS also for
 * flags other than a path or a schedule request; SSD_ERR_UNSUPPORTED for
 * another path or an unsupported shape); nothing is enqueued on error.
 * seqlen 0 passes the states through.  Enqueues on `stream` only; never
 * synchronises.
 */
ssd_status_t ssd_trap_scan_fwd(const void *v, const void *k, const void *q, const float *dt,
                               const float *a, const float *trap, const float *D,
                               const float *h0, const void *k0, const void *v0, void *y,
                               float *h_final, void *k_final, void *v_final,
                               const ssd_dims_t *dims, void *stream);

/*
 * ssd_conv1d_silu_fwd -- the causal depthwise conv1d + SiLU that precedes the
 * scan in the Mamba blocks of the pages (the builderforce Mamba2Block runs one
 * causal conv1d over the fused x, B and C projection channels; the conv1d
 * kernel page: y[b,t,d] = sum_k weight[d,k] x[b,t-k,d] + bias[d], zero before
 * the sequence; the mamba-rs 0.4.0 S6 forward applies SiLU in the same
 * kernel as the conv and carries the conv state from call to call).  Over
 * the fused channels c of xbc = [x (H*P) | B (G*N) | C (G*N)]:
 *   u[b,t,c] = SiLU(bias[c] + sum_{k<K} weight[c,k] xbc[b,t-k,c])
 * with xbc before t = 0 taken from conv_state (zero when NULL), and u written
 * split into the scan's x [B,L,H,P], B and C [B,L,G,N].
 *   xbc [B,L,C], conv_state and conv_state_out [B,K-1,C] (oldest step
 *     first) in dims->dtype; weight [C,K] and bias [C] (NULL: none) fp32.
 *   conv_state_out (NULL: not written) receives the last K-1 inputs, from
 *     which a following call continues; it must not overlap conv_state.
 * DEVICE pointers, 16-byte aligned, caller-owned; outputs overlap no input.
 * dims: batch, seqlen, nheads, headdim, dstate, ngroups, dtype as for
 * ssd_scan_fwd; chunk is ignored (>= 1); flags must be 0.  Supported:
 * kernel_size 2..4, H*P and G*N multiples of 8, batch <= 65535.  Errors as
 * ssd_scan_fwd (SSD_ERR_UNSUPPORTED for an unsupported size).  seqlen 0
 * passes the conv state through.  Enqueues on `stream` only.
 */
ssd_status_t ssd_conv1d_silu_fwd(const void *xbc, const float *weight, const float *bias,
                                 const void *conv_state, void *x, void *B, void *C,
                                 void *conv_state_out, int32_t kernel_size,
                                 const ssd_dims_t *dims, void *stream);

/*
 * ssd_conv_scan_fwd -- ssd_conv1d_silu_fwd followed by ssd_scan_fwd, in one call,
 * with the conv of the x channels done inside the chunked scan kernel (the
 * builderforce Mamba2Block runs the causal conv1d over the fused x, B, C
 * projection channels, then the SSD module, on one layer's buffers; the mamba-rs
 * 0.4.0 S6 forward carries the conv state between calls).  The scan reads the
 * raw x channels of xbc and applies the conv and SiLU to each tile in shared
 * memory, so the conv's x never goes through device memory; the B and C
 * channels (shared by every head of a group) are convolved once by a small
 * kernel beforehand.
 *   u = SiLU(conv(xbc)) split into x [B,L,H,P], B and C [B,L,G,N] as
 *   ssd_conv1d_silu_fwd defines it; then y, final_state as ssd_scan_fwd
 *   defines them for (x, dt_raw, dt_bias, A_log, B, C, D, init_state).
 * xbc [B,L,H*P + 2*G*N], conv_state and conv_state_out [B,K-1,H*P + 2*G*N]
 * (bf16); conv_weight [H*P + 2*G*N, K] and conv_bias (NULL: none) fp32;
 * kernel_size K in 2..4; the scan's arguments as for ssd_scan_fwd.  Nullable:
 * conv_bias, conv_state (zero), init_state (zero), final_state and
 * conv_state_out (not written).  DEVICE pointers of the current device,
 * caller-owned, 16-byte aligned; outputs overlap no input and each other
 * (conv_state_out must not overlap conv_state).
 * Supported: the chunked path's shapes (bf16, P = 64, N = 128, chunk % 64 == 0,
 * (H/G) even; GB300-class device); flags: SSD_PATH_AUTO or SSD_PATH_CHUNKED,
 * optionally a schedule request.  Scratch (the convolved B and C, and the
 * chunked path's) comes stream-ordered from the library pool.  Errors as
 * ssd_scan_fwd; SSD_ERR_UNSUPPORTED_DTYPE for fp32.  seqlen 0 passes both
 * states through.  Enqueues on `stream` only; never synchronises.
 */
ssd_status_t ssd_conv_scan_fwd(const void *xbc, const float *conv_weight, const float *conv_bias,
                               const void *conv_state, int32_t kernel_size, const float *dt_raw,
                               const float *dt_bias, const float *A_log, const float *D,
                               const float *init_state, void *y, float *final_state,
                               void *conv_state_out, const ssd_dims_t *dims, void *stream);

/*
 * ssd_gated_rmsnorm_fwd -- the gated output norm after the scan (the Mamba-3
 * forward of the pages, step F7 with its norm: RMSNorm(y) * weight * SiLU(z)),
 * per token over its H*P channels:
 *   out = y / sqrt(mean_c(y^2) + eps) * weight * SiLU(z)
 *   y, z, out [B,L,H,P] (dims->dtype); weight [H*P] fp32; eps >= 0.
 * DEVICE pointers, 16-byte aligned, caller-owned; out overlaps no input.
 * dims as for ssd_conv1d_silu_fwd (dstate, ngroups, chunk ignored beyond their
 * validation).  Supported: H*P a multiple of 8, at most 16384.  Errors as
 * ssd_scan_fwd.
 */
ssd_status_t ssd_gated_rmsnorm_fwd(const void *y, const void *z, const float *weight, float eps,
                                   void *out, const ssd_dims_t *dims, void *stream);

/*
 * ssd_complex_scan_fwd -- the complex-valued scan with exponential-trapezoidal
 * (ET) discretisation: the Mamba-3 complex SSD module of the pages, as its
 * header defines it (complex_ssd.ts).  Per batch row and head, with
 * A = exp(log|A| + i arg A) and dt_t = softplus(dt_raw_t + dt_bias):
 *   A_bar_t = exp(dt_t A),  B_bar_t = (A_bar_t - 1) A^-1 B_t  (the exact hold)
 *   h_t = A_bar_t h_{t-1} + B_bar_t x_t^T,  y_t = Re(C_t^T h_t) + D x_t
 * (The page's printed kernel exponentiates dt (log|A| + i arg A) and reads out
 * Re(conj(C) h); its header's statement is the one implemented.)
 * x, y [B,L,H,P] and B, C [B,L,G,N] in dims->dtype; B and C hold N/2 complex
 * numbers as (re, im) pairs along N; A_polar [H,2] fp32 = (log|A|, arg A);
 * dt_raw [B,L,H], dt_bias, D [H] fp32; init_state (NULL: zero) and
 * final_state (NULL: not written) [B,H,P,N] fp32, complex as (re, im) pairs
 * along N; final_state may be init_state (in place).  DEVICE pointers, 16-byte
 * aligned; y overlaps no input.  flags: SSD_PATH_SEQUENTIAL (one sequential
 * kernel; seqlen 1 is a decode step), SSD_PATH_CHUNKED (the chunk form on the
 * tensor cores: chunks of 64 steps, two batch rows per CTA, bf16 operands and
 * fp32 accumulation; bf16 with P = 64, N = 128 and seqlen >= 2 only, else
 * SSD_ERR_UNSUPPORTED) or SSD_PATH_AUTO (the chunk form where it applies, else
 * the sequential kernel).  The sequential kernel supports N % 4 == 0,
 * N <= 512; P <= 128 for N <= 128, P <= 64 for N <= 256, P <= 32 for
 * N <= 512; fp32 or bf16.  seqlen 0 copies the state through.  Errors as
 * ssd_scan_fwd.
 */
ssd_status_t ssd_complex_scan_fwd(const void *x, const float *dt_raw, const float *dt_bias,
                                  const float *A_polar, const void *B, const void *C, const float *D,
                                  const float *init_state, void *y, float *final_state,
                                  const ssd_dims_t *dims, void *stream);

/*
 * ssd_scan_bwd -- the backward of ssd_scan_fwd: the gradients of a loss with
 * respect to every input, given dy = dL/dy and d_final = dL/d final_state.
 * They are the derivatives of the recurrence ssd_scan_fwd evaluates (the
 * SSD module's forward, direct form).  The gradient of the state runs in
 * reverse:
 *   G_{L-1} = d_final + C_{L-1} dy_{L-1}^T,  G_t = dA_{t+1} G_{t+1} + C_t dy_t^T
 *   dx_t = D dy_t + dt_t G_t^T B_t,  dB_t = dt_t G_t x_t,  dC_t = h_t dy_t
 *   ddt_raw_t = sigmoid(dt_raw_t + dt_bias) sum G_t o (a dA_t h_{t-1} + B_t x_t^T)
 *   dA_log = a sum_t sum G_t o (dt_t dA_t h_{t-1}),  dD = sum_t dy_t . x_t,
 *   d_init = dA_0 G_0
 * with dB, dC summed over the heads of each group and the per-head gradients
 * over batch rows and steps, in a fixed order (deterministic).
 * Inputs as ssd_scan_fwd, plus dy [B,L,H,P] (dims->dtype) and d_final
 * [B,H,P,N] fp32 (NULL: zero).  Outputs, all fp32, caller-owned, overlapping
 * no input and each other: dx [B,L,H,P], ddt_raw [B,L,H], ddt_bias [H],
 * dA_log [H], dB and dC [B,L,G,N], dD [H], d_init [B,H,P,N] (NULL: not
 * written).  DEVICE pointers, 16-byte aligned.  flags: a path, plus
 * SSD_BWD_FP32_FORM and SSD_BWD_SPLIT_STATES (above).
 * SSD_PATH_CHUNKED: the chunk form (chunks of 64 steps in parallel: local
 * chunk states and state gradients, a pass over the chunks that links them,
 * then every gradient of a chunk as dense contractions); supported for
 * P <= 64, N <= 128, B*H <= 65535.  For bf16 with P = 64 and N = 128 its
 * contractions run on the tensor cores (bf16 operands, fp32 accumulation;
 * the chunk states enter as two bf16 terms), and the chunk states and their
 * links may be computed in one walk per (b, h) (SSD_BWD_SPLIT_STATES);
 * otherwise, or with SSD_BWD_FP32_FORM, as fp32 FFMA.  SSD_PATH_SEQUENTIAL: one sequential
 * kernel per (b, h) that recomputes the forward states segment by segment;
 * supported for N % 4 == 0, N <= 128, P <= 128.  SSD_PATH_AUTO takes the
 * chunk form where it applies, else the sequential kernel.  Scratch (chunk
 * states and gradients, or checkpoints; per-head gradients of B and C; the
 * per-head partial sums) comes stream-ordered from the library pool.  Errors
 * as ssd_scan_fwd.  Empty work writes nothing.
 */
ssd_status_t ssd_scan_bwd(const void *x, const float *dt_raw, const float *dt_bias, const float *A_log,
                          const void *B, const void *C, const float *D, const float *init_state,
                          const void *dy, const float *d_final, float *dx, float *ddt_raw,
                          float *ddt_bias, float *dA_log, float *dB, float *dC, float *dD,
                          float *d_init, const ssd_dims_t *dims, void *stream);

/* ---- the attention layers of hybrid state-space models ---------------------
 *
 * Hybrid stacks put a few attention layers between the scan layers.  The
 * operators below are such a layer's own: the step plan of a paged key-value
 * cache, the norm and rotary position of its queries and keys (forward, into
 * the cache when serving, and backward), and the attention that reads the
 * cache.  They have no counterpart in the cited pages; their formulas are in
 * the comments here.
 *
 * The paged cache.  Keys and values are kept in pages of page_size tokens.
 * Request r's token at position p lies in page block_table[r][p / page_size]
 * at offset p % page_size; its slot number is page * page_size + offset.
 * k_cache and v_cache are [npages, page_size, nkv, headdim] in dtype, addressed
 * by the strides given (elements) for page, token and head, headdim
 * contiguous: token-major and head-major pages and caches that share one
 * buffer are all covered.  Strides are multiples of 16 bytes.
 *
 * Arrays are DEVICE pointers of the current device, caller-owned.  Data
 * pointers are 16-byte aligned; positions, slots and the start array have
 * their type's alignment.  Queries, keys, values, their outputs and gradients,
 * and the two caches among themselves, may be views that interleave in one
 * buffer; an output that shares bytes with another operand is SSD_ERR_ALIASING,
 * but for the in-place forms named below.  Calls enqueue on `stream` only, never synchronise,
 * may be captured into a CUDA graph, and return an ssd_status_t; nothing is
 * enqueued on an argument error.
 */

typedef struct ssd_plan_dims {
    int64_t nreq;        /* requests: 0 .. SSD_PLAN_MAX_REQUESTS */
    int64_t max_tokens;  /* rows of positions, token_req and slots: 0 .. 2^31 - 1 */
    int64_t ring_size;   /* entries of free_ring: 1 .. 2^31 - 1 */
    int32_t page_size;   /* tokens per page, >= 1; page_size * max_pages <= 2^31 - 1 */
    int32_t max_pages;   /* columns of block_table (contiguous), >= 1 */
    uint32_t flags;      /* must be 0 */
    uint32_t reserved;   /* must be 0 */
} ssd_plan_dims_t;

#define SSD_PLAN_MAX_REQUESTS 8192

/*
 * ssd_paged_plan -- block tables, positions and slots of one serving step.
 *
 * Request r holds lens[r] cached tokens (in ceil(lens[r] / page_size) pages of
 * its block_table row) and brings new_lens[r] tokens: 0 none, < 0 the request
 * is finished and gives its pages back.  Free pages are the ring entries
 * free_ring[i mod ring_size], ring_pos[0] <= i < ring_pos[1].
 * In request order: a request that brings tokens is granted all of them if
 * lens + new_lens fits its table row and the tokens and the new pages of it
 * and of all requests before it (that fit their rows) are at most max_tokens
 * and the free pages; else it is granted none and keeps its state.  So the
 * first request that finds no room and every later one wait.  Granted
 * requests take their pages from the ring's head, in request order, into
 * their block_table rows; finished ones put theirs at its tail, in request
 * order, to be handed out from the next call on.
 *   lens_out [nreq]   lens + granted; 0 for a finished request
 *   granted  [nreq]   new_lens or 0
 *   start    [nreq+1] exclusive prefix sum of granted: request r's tokens are
 *                     rows start[r] .. start[r+1] - 1 of the step
 *   positions, token_req, slots [max_tokens]  per row, -1 beyond start[nreq]
 *   ring_pos_out [2]  the ring's head and tail afterwards
 *   counts   [4]      tokens granted, pages taken, pages given back, requests
 *                     refused
 * lens_out may be lens and ring_pos_out may be ring_pos (in place); nothing
 * else may overlap.  block_table rows change only in the entries of new
 * pages.  A negative len counts as 0; a ring with fewer than 0 or more than
 * ring_size free entries counts as one with 0 or ring_size.  Pointers are
 * 16-byte aligned; the arrays of max_tokens entries may be NULL when it is 0.
 */
ssd_status_t ssd_paged_plan(const int32_t *lens, const int32_t *new_lens, int32_t *block_table,
                            int32_t *free_ring, const int64_t *ring_pos, int32_t *lens_out,
                            int32_t *granted, int32_t *start, int32_t *positions,
                            int32_t *token_req, int64_t *slots, int64_t *ring_pos_out,
                            int32_t *counts, const ssd_plan_dims_t *dims, void *stream);

/* In ssd_qk_dims_t.flags: rotated pairs are the adjacent elements (2i, 2i+1);
 * without it they are (i, i + rotary_dim / 2). */
#define SSD_ROPE_INTERLEAVED 1u

typedef struct ssd_qk_dims {
    int64_t ntokens;     /* >= 0; times either number of heads at most 2^30 */
    int64_t max_pos;     /* rows of cos and sin, >= 0 */
    int64_t npages;      /* pages of the cache (0 without one) */
    int32_t nheads_q;    /* >= 1 */
    int32_t nheads_k;    /* >= 1; also the heads of v */
    int32_t headdim;     /* D: a multiple of 8, 8 .. 256 */
    int32_t rotary_dim;  /* R: a multiple of 16, 0 .. D; the elements from R on are not rotated */
    int32_t page_size;   /* >= 1 with a cache */
    int32_t dtype;       /* ssd_dtype_t of q, k, v, their outputs and gradients, and the cache */
    uint32_t flags;      /* 0 or SSD_ROPE_INTERLEAVED */
    float eps;           /* >= 0 */
    /* strides in elements, {token, head}, D contiguous; multiples of 16 bytes */
    int64_t q_stride[2], k_stride[2], v_stride[2];
    int64_t qo_stride[2], ko_stride[2];   /* q_out, k_out; in the backward dq_out, dk_out */
    int64_t dq_stride[2], dk_stride[2];   /* backward only */
    /* strides in elements, {page, token, head} */
    int64_t kc_stride[3], vc_stride[3];
} ssd_qk_dims_t;

/*
 * ssd_qk_norm_rope_fwd -- per token and head, RMSNorm of the queries and keys
 * over the head's D elements, then the rotary position:
 *   n = x / sqrt(mean(x^2) + eps) * weight
 *   (a, b) -> (a cos - b sin, b cos + a sin) for each rotated pair of n
 * with cos and sin [max_pos, R/2] fp32 taken at the token's position; computed
 * in fp32 and rounded once.  A row of zeros stays zero, with eps 0 too (its
 * gradient is zero then, and it has no part in the weights').  Inputs q
 * [ntokens, Hq, D], k [ntokens, Hk, D], q_weight and k_weight [D] fp32 (NULL:
 * ones), positions [ntokens].  Outputs q_out, k_out (k_out may be NULL when
 * there is a cache).
 * With k_cache (then v, v_cache and slots are required too): token t's keys
 * and its v [ntokens, Hk, D], unchanged, are also written to slot slots[t] of
 * the caches; a slot outside 0 .. npages * page_size - 1 is not written.
 * A token whose position is outside 0 .. max_pos - 1 is padding: its q_out and
 * k_out are zero and nothing of it goes to the cache.
 * q_out may be q, and k_out k, with equal strides (in place); outputs overlap
 * no other input.  The caches' rows are distinct memory, and the two caches may
 * be views of one buffer but share no bytes.  Two tokens of a call must not have
 * the same slot.
 */
ssd_status_t ssd_qk_norm_rope_fwd(const void *q, const void *k, const void *v,
                                  const float *q_weight, const float *k_weight,
                                  const float *cos, const float *sin, const int32_t *positions,
                                  void *q_out, void *k_out, void *k_cache, void *v_cache,
                                  const int64_t *slots, const ssd_qk_dims_t *dims, void *stream);

/*
 * ssd_qk_norm_rope_bwd -- the gradients of ssd_qk_norm_rope_fwd with respect
 * to q, k and the weights, given dq_out = dL/dq_out and dk_out = dL/dk_out.
 * With g the inversely rotated gradient, r = 1 / sqrt(mean(x^2) + eps):
 *   dweight = sum over tokens and heads of g x r   (fp32, a fixed order)
 *   dx = r (g weight - x r mean(g weight x r))
 * dq, dk in dtype; dq_weight, dk_weight [D] fp32 (NULL: not written).  Padding
 * tokens have zero dq, dk and no part in the weights' gradients.  Outputs
 * overlap no input, except that dq may be dq_out and dk dk_out with equal
 * strides.  `workspace`: NULL (scratch comes stream-ordered from the library
 * pool), or a 16-byte aligned buffer of workspace_bytes >= the size that
 * ssd_qk_norm_rope_bwd_workspace_size gives (else SSD_ERR_SCRATCH_LIMIT),
 * which calls that may overlap must not share; its contents do not matter.
 */
ssd_status_t ssd_qk_norm_rope_bwd(const void *q, const void *k, const float *q_weight,
                                  const float *k_weight, const float *cos, const float *sin,
                                  const int32_t *positions, const void *dq_out,
                                  const void *dk_out, void *dq, void *dk, float *dq_weight,
                                  float *dk_weight, void *workspace, uint64_t workspace_bytes,
                                  const ssd_qk_dims_t *dims, void *stream);
ssd_status_t ssd_qk_norm_rope_bwd_workspace_size(const ssd_qk_dims_t *dims, uint64_t *bytes);

#define SSD_ATTN_MAX_REQUESTS 16384

typedef struct ssd_attn_dims {
    int64_t nrows;       /* query rows (tokens), >= 0 */
    int64_t nreq;        /* requests: rows of block_table, >= 0 */
    int64_t npages;      /* pages of the cache, >= 0 */
    int32_t nheads;      /* query heads, >= 1 */
    int32_t nkv;         /* key-value heads, >= 1, nheads % nkv == 0; query head h reads head h / (nheads / nkv) */
    int32_t headdim;     /* D: a multiple of 8, 8 .. 256 */
    int32_t page_size;   /* >= 1; page_size * max_pages <= 2^31 - 1 */
    int32_t max_pages;   /* columns of block_table, >= 1 */
    int32_t window;      /* 0: none; else a row sees its last `window` positions only */
    int32_t dtype;       /* ssd_dtype_t of q, the caches and out */
    uint32_t flags;      /* must be 0 */
    float scale;         /* factor of q . k */
    uint32_t reserved;   /* must be 0 */
    /* strides in elements, D contiguous; multiples of 16 bytes (table_stride: any) */
    int64_t q_stride[2], o_stride[2];     /* row, head */
    int64_t kc_stride[3], vc_stride[3];   /* page, token, head; the first two below 2^32 x 16 bytes (else SSD_ERR_UNSUPPORTED) */
    int64_t table_stride;                 /* request */
} ssd_attn_dims_t;

/*
 * ssd_paged_attn_fwd -- attention of new tokens over a paged cache.
 *
 * Row i is the token at position positions[i] of its request and sees the
 * cached positions t with max(0, positions[i] - window + 1) <= t <=
 * positions[i] (all from 0 without a window):
 *   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t e^{s_t}
 * start NULL: row i is request i's one row (nrows == nreq).  Else start
 * [nreq+1], ascending, as ssd_paged_plan writes it: request r has the rows
 * start[r] .. start[r+1] - 1, their positions ascending; rows from
 * start[nreq] on are padding.  nreq <= SSD_ATTN_MAX_REQUESTS then.
 * A row that sees nothing (a negative position, padding) has out 0 and lse
 * -inf.  Infinities and NaN among the values that a row sees give what the sum
 * gives.  However large finite scores are, weights come from their differences.
 * Positions past max_pages * page_size, and pages whose table entry is outside
 * 0 .. npages - 1, are not seen; table entries past a request's positions are not
 * read into the result, and neither are cache contents that a row does not
 * see, whatever they hold (infinities and NaN included).
 * q, out [nrows, nheads, D]; lse [nrows, nheads] fp32 (NULL: not written);
 * block_table [nreq, max_pages].  Sums, maxima and the accumulated output are
 * fp32.  The work is split over the cache's length into equal shares and
 * joined in a fixed order: equal calls on one device give equal bits.
 * out may be q with equal strides; outputs overlap no other input.
 * `workspace` as for ssd_qk_norm_rope_bwd, with
 * ssd_paged_attn_workspace_size's bytes.
 */
ssd_status_t ssd_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_table, const int32_t *positions,
                                const int32_t *start, void *out, float *lse, void *workspace,
                                uint64_t workspace_bytes, const ssd_attn_dims_t *dims,
                                void *stream);
ssd_status_t ssd_paged_attn_workspace_size(const ssd_attn_dims_t *dims, uint64_t *bytes);

/*
 * ---------------------------------------------------------------------------
 * One layer's step around the scan: the norm in front with the residual's
 * addition, products of 8-bit integers for the two projections, the gated norm
 * into 8 bits, and the convolution and scan for single tokens.
 *
 * Rows are [rows, dim] with a stride between rows (elements; dim contiguous).
 * An 8-bit row is a row of whole numbers q, -127 .. 127, with one fp32 scale:
 * it stands for q * scale, scale = max|v| / 127 and q = v / scale rounded to
 * nearest even.  A row of zeros has scale 0, and a row that holds an infinity or
 * NaN has q 0 and scale NaN, so that whatever is computed from it is NaN.  The
 * ends of the range: v is r times t = h * weight (* SiLU(z)), r one factor a row, and
 * t is formed in fp32.  A row whose largest |t|, or whose scale, is below 2^-126
 * has scale 0; one where t leaves fp32's range is taken to hold an infinity.
 *
 * Pointers and errors as for the attention-layer entry points: DEVICE arrays of
 * the current device, 16-byte aligned where nothing else is said; calls enqueue
 * on `stream` only, never synchronise, may be captured into a CUDA graph;
 * nothing is enqueued on an argument error.
 */

typedef struct ssd_norm_dims {
    int64_t rows;            /* >= 0, below 2^31 */
    int32_t dim;             /* D: a multiple of 8, 8 .. 16384 */
    int32_t dtype;           /* ssd_dtype_t of x, out (and y, z; dout) */
    int32_t residual_dtype;  /* ssd_dtype_t of residual and residual_out (h, dresidual and dx): dtype or SSD_DTYPE_F32 */
    uint32_t flags;          /* must be 0 */
    float eps;               /* >= 0 */
    uint32_t reserved;       /* must be 0 */
    /* row strides in elements, multiples of 16 bytes (q_stride: of 8; z_stride: any); inputs 0 or more (rows may
     * share bytes), outputs at least dim; not looked at where there is one row */
    int64_t x_stride;        /* x; y; in the backward dout */
    int64_t z_stride;        /* z */
    int64_t residual_stride; /* residual; in the backward dresidual */
    int64_t out_stride;      /* out; in the backward dx */
    int64_t ro_stride;       /* residual_out; in the backward h */
    int64_t q_stride;        /* q */
} ssd_norm_dims_t;

/*
 * ssd_add_rmsnorm_fwd -- the residual's addition and RMSNorm, per row:
 *   h = x + residual,   v = h / sqrt(mean(h^2) + eps) * weight
 * computed in fp32 from the sum before it is rounded.  Outputs, each rounded
 * once: residual_out = h (residual_dtype), out = v (dtype), or v as an 8-bit row
 * in q [rows, D] and q_scale [rows].  Exactly one of out and q is given, q_scale
 * with q.  residual NULL: h = x, and residual_out has to be NULL too; with a
 * residual, residual_out may be NULL.  weight [D] fp32.  A row of zeros stays
 * zero, with eps 0 too.  The mean square is an fp32 sum: where it overflows (values
 * near 2^64), the row is normalised to zeros.  With eps 0, values below about
 * 2^-63 have squares that lose bits, and a row of values below 2^-75 counts as zeros.
 * residual_out may be residual with equal strides, and out may be x (in place);
 * nothing else may overlap.
 */
ssd_status_t ssd_add_rmsnorm_fwd(const void *x, const void *residual, const float *weight,
                                 void *out, int8_t *q, float *q_scale, void *residual_out,
                                 const ssd_norm_dims_t *dims, void *stream);

/*
 * ssd_add_rmsnorm_bwd -- the gradients of ssd_add_rmsnorm_fwd (out in dtype).
 * h is what the forward wrote as residual_out (without a residual: x), dout =
 * dL/dout, dresidual = dL/dresidual_out (NULL: none).  With
 * r = 1 / sqrt(mean(h^2) + eps) and g = dout weight:
 *   dx = r (g - h r^2 mean(g h)) + dresidual   (of x and of residual alike)
 *   dweight = sum over rows of dout h r        (fp32, a fixed order)
 * h, dresidual and dx are in residual_dtype, dout in dtype.  dweight [D] fp32
 * (NULL: not written).  A row of zeros with eps 0 has r = 0, and so has
 * one whose mean square overflows (its dx is dresidual; NaN where the sum of g h
 * overflows too, with values near 2^120).  dx may be
 * dresidual, or dout where the types are the same (equal strides, in place);
 * outputs overlap nothing else.  `workspace` as for ssd_qk_norm_rope_bwd, with
 * ssd_add_rmsnorm_bwd_workspace_size's bytes.
 */
ssd_status_t ssd_add_rmsnorm_bwd(const void *h, const float *weight, const void *dout,
                                 const void *dresidual, void *dx, float *dweight,
                                 void *workspace, uint64_t workspace_bytes,
                                 const ssd_norm_dims_t *dims, void *stream);
ssd_status_t ssd_add_rmsnorm_bwd_workspace_size(const ssd_norm_dims_t *dims, uint64_t *bytes);

/*
 * ssd_gated_rmsnorm_q8_fwd -- ssd_gated_rmsnorm_fwd with an 8-bit result:
 *   v = y / sqrt(mean(y^2) + eps) * weight * SiLU(z)
 * as an 8-bit row in q [rows, D] and q_scale [rows].  y and z [rows, D] in
 * dtype, weight [D] fp32.  z may have any alignment of its type (a slice of the
 * projection's rows).  Outputs overlap nothing.
 */
ssd_status_t ssd_gated_rmsnorm_q8_fwd(const void *y, const void *z, const float *weight,
                                      int8_t *q, float *q_scale, const ssd_norm_dims_t *dims,
                                      void *stream);

/* Weights of ssd_q8_matmul are kept in the order that it reads them: tiles of
 * 128 output channels; in a tile, for each 16 inner elements, the 128 channels'
 * 16 bytes side by side (byte ((tile * K64 * 4 + k / 16) * 128 + n % 128) * 16 +
 * k % 16 with tile = n / 128 and K64 = ceil(K / 64)); zeros beyond N and K. */
#define SSD_Q8_PACKED_BYTES(N, K) ((((int64_t)(N) + 127) / 128 * 128) * (((int64_t)(K) + 63) / 64 * 64))

typedef struct ssd_q8_dims {
    int64_t M;           /* tokens, >= 0, below 2^31 */
    int32_t N;           /* output channels, 1 .. 2^24 */
    int32_t K;           /* inner elements, 1 .. 65536 */
    int32_t out_dtype;   /* ssd_dtype_t of y */
    uint32_t flags;      /* must be 0 */
    int64_t a_stride;    /* row strides in elements: a any from 0 up (rows may share bytes), y any >= N; */
                         /* ssd_q8_pack_weight: the weight's, >= K */
    int64_t y_stride;
} ssd_q8_dims_t;

/* ssd_q8_pack_weight -- w [N, K] (rows a_stride apart) into `packed`, SSD_Q8_PACKED_BYTES(N, K)
 * bytes.  M, out_dtype and y_stride are not looked at.  w may have any alignment. */
ssd_status_t ssd_q8_pack_weight(const int8_t *w, int8_t *packed, const ssd_q8_dims_t *dims, void *stream);

/*
 * ssd_q8_matmul -- products of 8-bit integers:
 *   y[t, n] = (sum_k a[t, k] w[n, k]) * a_scale[t] * w_scale[n]
 * a [M, K] int8 (all values -128 .. 127), w packed, a_scale [M], w_scale [N] fp32,
 * y [M, N] in out_dtype.  The sum is exact whatever its order, so a row's result
 * does not depend on the other rows or on how the work was split; it is
 * rounded to fp32, multiplied by a_scale, then by w_scale, and rounded to
 * out_dtype.  a and y have any alignment of their types, the scales 4 bytes.
 * y overlaps nothing.  `workspace` as for ssd_qk_norm_rope_bwd, with
 * ssd_q8_matmul_workspace_size's bytes:
 *   M <= 8:    none
 *   M <= 256:  128 ceil(M / 128) * 128 ceil(K / 64), the tokens in 16 bits
 *   above:     16384 ceil(K / 64) (ceil(N / 128) + ceil(min(M, 32768) / 128)) + 32768, the weights
 *              in 16 bits (about 2 N K bytes, whatever M is) and up to 32768 tokens at a time
 */
ssd_status_t ssd_q8_matmul(const int8_t *a, const float *a_scale, const int8_t *packed,
                           const float *w_scale, void *y, void *workspace,
                           uint64_t workspace_bytes, const ssd_q8_dims_t *dims, void *stream);
ssd_status_t ssd_q8_matmul_workspace_size(const ssd_q8_dims_t *dims, uint64_t *bytes);

typedef struct ssd_step_dims {
    int64_t rows;        /* tokens of the step, >= 0; rows * nheads below 2^31 */
    int64_t nslots;      /* sequences that conv_ring and states hold, >= 0 */
    int32_t nheads;      /* H: 1 .. 2^20 */
    int32_t headdim;     /* P: 1 .. 2048 */
    int32_t dstate;      /* N: a multiple of 4, 4 .. 512 */
    int32_t ngroups;     /* G >= 1, H % G == 0; C = H P + 2 G N below 2^30 */
    int32_t kernel_size; /* K: 2 .. 4 */
    int32_t dtype;       /* ssd_dtype_t of xbc, conv_ring and y */
    int32_t dt_dtype;    /* ssd_dtype_t of dt_raw: dtype or SSD_DTYPE_F32 */
    uint32_t flags;      /* must be 0 */
    /* row strides in elements; inputs any from 0 up (rows may share bytes) */
    int64_t xbc_stride;
    int64_t dt_stride;
    int64_t y_stride;    /* >= H P */
} ssd_step_dims_t;

/*
 * ssd_conv_scan_step -- ssd_conv_scan_fwd for one token of each of several
 * sequences, their states in a pool.
 *
 * Row i is the token at position t = positions[i] of the sequence in slot s =
 * slots[i].  conv_ring [nslots, K, C] holds each sequence's last K inputs, that
 * of position p in entry p mod K.  With the K-1 inputs before it (zeros before
 * position 0) and its own xbc[i]:
 *   u = SiLU(bias + sum_j weight[:, j] input(t - j)),   x | B | C = u
 *   h = exp(dt A) h + dt B x^T,   y[i] = C^T h + D x
 * with dt = softplus(dt_raw[i] + dt_bias), A = -exp(A_log) and h = states[s]
 * [H, P, N] fp32, updated in place; xbc[i] goes into the ring's entry t mod K.  At
 * position 0 a sequence begins: neither the ring nor the state of the slot is
 * read.  x, B and C are kept in fp32 between the convolution and the scan.
 * A row with a slot outside 0 .. nslots - 1 or a negative position is padding: its
 * y is zero and nothing is written for it.  Two rows must not have the same slot.
 * xbc [rows, C], dt_raw [rows, H], y [rows, H P]; weight [C, K], bias [C] (NULL:
 * none), dt_bias, A_log, D [H] fp32; slots and positions [rows] int32.  xbc, dt_raw
 * and y have any alignment of their types, the [H] arrays, bias, slots and
 * positions 4 bytes.  Outputs overlap nothing.
 */
ssd_status_t ssd_conv_scan_step(const void *xbc, void *conv_ring, const float *weight,
                                const float *bias, const void *dt_raw, const float *dt_bias,
                                const float *A_log, const float *D, float *states,
                                const int32_t *slots, const int32_t *positions, void *y,
                                const ssd_step_dims_t *dims, void *stream);

/* Which path SSD_PATH_AUTO resolves to for these dims on the current device
 * (SSD_PATH_SEQUENTIAL, SSD_PATH_CHUNKED or SSD_PATH_DECODE), or
 * -(ssd_status_t) if the dims are
 * invalid or unsupported.  Host only; launches nothing. */
int32_t ssd_select_path(const ssd_dims_t *dims);

/* Kernel launches one ssd_scan_fwd call makes for these dims (0 for empty
 * work), or -(ssd_status_t).  Host only. */
int32_t ssd_launches_per_call(const ssd_dims_t *dims);

/* How the chunked path orders its work for these dims and flags on the
 * current device (the SM count enters the choice), as ssd_scan_fwd would run
 * it:
 *   SSD_SCHEDULE_NONE    no chunked work (empty, or the sequential path);
 *   SSD_SCHEDULE_RANGES  chains cut into units of whole chunks, dealt to the CTAs
 *                        in turn; a unit takes its entering state from the unit
 *                        before it in its chain (one launch);
 *   SSD_SCHEDULE_PIECES  the chains' 128-step sub-chunks, chain after chain, cut
 *                        into one run of equal length per CTA; a chain cut
 *                        between two CTAs hands its state across (one launch);
 *   SSD_SCHEDULE_SPLIT   units of whole chunks or (where a chunk is a whole
 *                        number of 128-step sub-chunks) of whole sub-chunks:
 *                        every unit's end state from zero, a combine of those
 *                        states along each chain, then every unit from its
 *                        combined entering state (three launches; two where a
 *                        chain has at most 4 units and the scan has no conv or
 *                        trapezoidal mode: each unit then combines its
 *                        predecessors' end states itself).
 * All three evaluate the chunked recurrence with the state carried from chunk
 * to chunk; they differ only in which CTA computes what, and when.
 * ssd_scan_fwd_noalloc may choose differently (see there).  Returns -(ssd_status_t)
 * for invalid or unsupported dims.  Host only; launches nothing. */
int32_t ssd_chunk_schedule(const ssd_dims_t *dims);

/* Total kernel launches this library has made in this process. */
uint64_t ssd_launch_count(void);

/* Synchronises `stream`, then reads and clears the device error word of the
 * current device into *code (0 = none, else an ssd_status_t such as
 * SSD_ERR_TIMEOUT).  Returns SSD_OK, or SSD_ERR_CUDA if the read failed. */
ssd_status_t ssd_get_device_error(void *stream, uint32_t *code);

/* Static description of a status code.  Never NULL (an unknown value gives
 * "unknown status"). */
const char *ssd_status_string(ssd_status_t status);

/* SSD_ABI_VERSION of the loaded library. */
int32_t ssd_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBSSD_SSD_H */
