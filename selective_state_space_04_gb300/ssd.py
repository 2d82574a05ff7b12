"""ctypes binding for libssd (argument marshalling only).

Every step of the scan runs in libssd's CUDA kernels.  If the shared library
has not been built, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

PATH_AUTO = 0
DIAG_STALL_HANDOFF = 0x100
BWD_FP32_FORM = 0x200   # ssd_scan_bwd: the chunk form's fp32 contractions even where the tensor-core pass applies
BWD_SPLIT_STATES = 0x400   # ssd_scan_bwd: the tensor-core form's chunk states and chains as two launches
PATH_SEQUENTIAL = 1
PATH_CHUNKED = 2
PATH_DECODE = 3
_PATHS = {"auto": PATH_AUTO, "sequential": PATH_SEQUENTIAL, "seq": PATH_SEQUENTIAL,
          "chunked": PATH_CHUNKED, "decode": PATH_DECODE}

DTYPE_F32 = 0
DTYPE_BF16 = 1

STATUS = {0: "SSD_OK", 1: "SSD_ERR_INVALID_DIMS", 2: "SSD_ERR_NULL_PTR", 3: "SSD_ERR_MISALIGNED",
          4: "SSD_ERR_UNSUPPORTED", 5: "SSD_ERR_CUDA", 6: "SSD_ERR_TIMEOUT", 7: "SSD_ERR_ALIASING",
          8: "SSD_ERR_SCRATCH_LIMIT", 9: "SSD_ERR_UNSUPPORTED_DTYPE"}


class SsdError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {what}")


class SsdDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class SsdPlanDims(ctypes.Structure):
    _fields_ = [("nreq", ctypes.c_int64), ("max_tokens", ctypes.c_int64), ("ring_size", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


ROPE_INTERLEAVED = 1


class SsdQkDims(ctypes.Structure):
    _fields_ = [("ntokens", ctypes.c_int64), ("max_pos", ctypes.c_int64), ("npages", ctypes.c_int64),
                ("nheads_q", ctypes.c_int32), ("nheads_k", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
                ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2),
                ("qo_stride", ctypes.c_int64 * 2), ("ko_stride", ctypes.c_int64 * 2),
                ("dq_stride", ctypes.c_int64 * 2), ("dk_stride", ctypes.c_int64 * 2),
                ("kc_stride", ctypes.c_int64 * 3), ("vc_stride", ctypes.c_int64 * 3)]


class SsdAttnDims(ctypes.Structure):
    _fields_ = [("nrows", ctypes.c_int64), ("nreq", ctypes.c_int64), ("npages", ctypes.c_int64),
                ("nheads", ctypes.c_int32), ("nkv", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("window", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_uint32),
                ("q_stride", ctypes.c_int64 * 2), ("o_stride", ctypes.c_int64 * 2),
                ("kc_stride", ctypes.c_int64 * 3), ("vc_stride", ctypes.c_int64 * 3), ("table_stride", ctypes.c_int64)]


class SsdNormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_uint32), ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("ro_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64)]


class SsdQ8Dims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("a_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]


class SsdStepDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("nslots", ctypes.c_int64), ("nheads", ctypes.c_int32),
                ("headdim", ctypes.c_int32), ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("kernel_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("dt_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("xbc_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64)]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libssd is not built ({path} missing); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, fp = ctypes.c_void_p, ctypes.c_void_p
    sig = [vp, fp, fp, fp, vp, vp, fp, fp, vp, fp, ctypes.POINTER(SsdDims), vp]
    for name in ("ssd_scan_fwd", "ssd_scan_fwd_host", "ssd_scan_fwd_noalloc"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = sig
    lib.ssd_scan_fwd_ws.restype = ctypes.c_int
    lib.ssd_scan_fwd_ws.argtypes = sig[:10] + [vp, ctypes.c_uint64, ctypes.POINTER(SsdDims), vp]
    lib.ssd_scan_fwd_workspace_size.restype = ctypes.c_int
    lib.ssd_scan_fwd_workspace_size.argtypes = [ctypes.POINTER(SsdDims), ctypes.POINTER(ctypes.c_uint64)]
    lib.ssd_select_path.restype = ctypes.c_int32
    lib.ssd_select_path.argtypes = [ctypes.POINTER(SsdDims)]
    lib.ssd_launches_per_call.restype = ctypes.c_int32
    lib.ssd_launches_per_call.argtypes = [ctypes.POINTER(SsdDims)]
    lib.ssd_chunk_schedule.restype = ctypes.c_int32
    lib.ssd_chunk_schedule.argtypes = [ctypes.POINTER(SsdDims)]
    lib.ssd_launch_count.restype = ctypes.c_uint64
    lib.ssd_launch_count.argtypes = []
    lib.ssd_get_device_error.restype = ctypes.c_int
    lib.ssd_get_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [ctypes.c_int32]
    lib.ssd_abi_version.restype = ctypes.c_int32
    lib.ssd_abi_version.argtypes = []
    lib.ssd_trap_scan_fwd.restype = ctypes.c_int
    lib.ssd_trap_scan_fwd.argtypes = [vp] * 14 + [ctypes.POINTER(SsdDims), vp]
    lib.ssd_conv1d_silu_fwd.restype = ctypes.c_int
    lib.ssd_conv1d_silu_fwd.argtypes = [vp] * 8 + [ctypes.c_int32, ctypes.POINTER(SsdDims), vp]
    lib.ssd_conv_scan_fwd.restype = ctypes.c_int
    lib.ssd_conv_scan_fwd.argtypes = [vp] * 4 + [ctypes.c_int32] + [vp] * 8 + [ctypes.POINTER(SsdDims), vp]
    lib.ssd_gated_rmsnorm_fwd.restype = ctypes.c_int
    lib.ssd_gated_rmsnorm_fwd.argtypes = [vp, vp, vp, ctypes.c_float, vp, ctypes.POINTER(SsdDims), vp]
    lib.ssd_scan_bwd.restype = ctypes.c_int
    lib.ssd_scan_bwd.argtypes = [vp] * 18 + [ctypes.POINTER(SsdDims), vp]
    lib.ssd_complex_scan_fwd.restype = ctypes.c_int
    lib.ssd_complex_scan_fwd.argtypes = [vp] * 10 + [ctypes.POINTER(SsdDims), vp]
    lib.ssd_paged_plan.restype = ctypes.c_int
    lib.ssd_paged_plan.argtypes = [vp] * 13 + [ctypes.POINTER(SsdPlanDims), vp]
    lib.ssd_qk_norm_rope_fwd.restype = ctypes.c_int
    lib.ssd_qk_norm_rope_fwd.argtypes = [vp] * 13 + [ctypes.POINTER(SsdQkDims), vp]
    lib.ssd_qk_norm_rope_bwd.restype = ctypes.c_int
    lib.ssd_qk_norm_rope_bwd.argtypes = [vp] * 14 + [ctypes.c_uint64, ctypes.POINTER(SsdQkDims), vp]
    lib.ssd_qk_norm_rope_bwd_workspace_size.restype = ctypes.c_int
    lib.ssd_qk_norm_rope_bwd_workspace_size.argtypes = [ctypes.POINTER(SsdQkDims), ctypes.POINTER(ctypes.c_uint64)]
    lib.ssd_paged_attn_fwd.restype = ctypes.c_int
    lib.ssd_paged_attn_fwd.argtypes = [vp] * 9 + [ctypes.c_uint64, ctypes.POINTER(SsdAttnDims), vp]
    lib.ssd_paged_attn_workspace_size.restype = ctypes.c_int
    lib.ssd_paged_attn_workspace_size.argtypes = [ctypes.POINTER(SsdAttnDims), ctypes.POINTER(ctypes.c_uint64)]
    lib.ssd_add_rmsnorm_fwd.restype = ctypes.c_int
    lib.ssd_add_rmsnorm_fwd.argtypes = [vp] * 7 + [ctypes.POINTER(SsdNormDims), vp]
    lib.ssd_gated_rmsnorm_q8_fwd.restype = ctypes.c_int
    lib.ssd_gated_rmsnorm_q8_fwd.argtypes = [vp] * 5 + [ctypes.POINTER(SsdNormDims), vp]
    lib.ssd_add_rmsnorm_bwd.restype = ctypes.c_int
    lib.ssd_add_rmsnorm_bwd.argtypes = [vp] * 7 + [ctypes.c_uint64, ctypes.POINTER(SsdNormDims), vp]
    lib.ssd_add_rmsnorm_bwd_workspace_size.restype = ctypes.c_int
    lib.ssd_add_rmsnorm_bwd_workspace_size.argtypes = [ctypes.POINTER(SsdNormDims), ctypes.POINTER(ctypes.c_uint64)]
    lib.ssd_q8_pack_weight.restype = ctypes.c_int
    lib.ssd_q8_pack_weight.argtypes = [vp] * 2 + [ctypes.POINTER(SsdQ8Dims), vp]
    lib.ssd_q8_matmul.restype = ctypes.c_int
    lib.ssd_q8_matmul.argtypes = [vp] * 6 + [ctypes.c_uint64, ctypes.POINTER(SsdQ8Dims), vp]
    lib.ssd_q8_matmul_workspace_size.restype = ctypes.c_int
    lib.ssd_q8_matmul_workspace_size.argtypes = [ctypes.POINTER(SsdQ8Dims), ctypes.POINTER(ctypes.c_uint64)]
    lib.ssd_conv_scan_step.restype = ctypes.c_int
    lib.ssd_conv_scan_step.argtypes = [vp] * 12 + [ctypes.POINTER(SsdStepDims), vp]
    return lib


_lib = load_library()


def lib() -> ctypes.CDLL:
    return _lib


SCHEDULE_SHIFT = 4
_SCHEDULE_REQUESTS = {"auto": 0, "ranges": 1, "pieces": 2, "split": 3}


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, dtype, path="auto",
              schedule="auto") -> SsdDims:
    d = SsdDims()
    d.batch, d.seqlen, d.nheads, d.headdim = batch, seqlen, nheads, headdim
    d.dstate, d.ngroups, d.chunk = dstate, ngroups, chunk
    if isinstance(dtype, int):     # an ssd_dtype_t value, passed through as given
        d.dtype = dtype
    else:
        d.dtype = DTYPE_BF16 if dtype in ("bf16", torch.bfloat16) else DTYPE_F32
    d.flags = (_PATHS[path] if isinstance(path, str) else int(path)) | \
        (_SCHEDULE_REQUESTS[schedule] << SCHEDULE_SHIFT)
    d.reserved = 0
    return d


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str):
    if status != 0:
        raise SsdError(status, what)


def _dims_from(x, B, chunk, path, schedule="auto"):
    Bt, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return make_dims(Bt, L, H, P, N, G, chunk, x.dtype, path, schedule)


def select_path(x_shape, ngroups, dstate, chunk, dtype="bf16", path="auto", schedule="auto") -> int:
    Bt, L, H, P = x_shape
    d = make_dims(Bt, L, H, P, dstate, ngroups, chunk, dtype, path, schedule)
    return _lib.ssd_select_path(ctypes.byref(d))


def launches_per_call(x_shape, ngroups, dstate, chunk, dtype="bf16", path="auto", schedule="auto") -> int:
    Bt, L, H, P = x_shape
    d = make_dims(Bt, L, H, P, dstate, ngroups, chunk, dtype, path, schedule)
    return _lib.ssd_launches_per_call(ctypes.byref(d))


SCHEDULES = {0: "none", 1: "ranges", 2: "pieces", 3: "split"}


def chunk_schedule(x_shape, ngroups, dstate, chunk, dtype="bf16", path="auto", schedule="auto") -> str:
    """How ``ssd_scan_fwd`` orders the chunked path's work for these sizes on the current device."""
    Bt, L, H, P = x_shape
    d = make_dims(Bt, L, H, P, dstate, ngroups, chunk, dtype, path, schedule)
    v = _lib.ssd_chunk_schedule(ctypes.byref(d))
    if v < 0:
        _check(-v, "ssd_chunk_schedule")
    return SCHEDULES[v]


def workspace_size(x_shape, ngroups, dstate, chunk, dtype="bf16", path="auto", schedule="auto") -> int:
    """Bytes of scratch ``ssd_scan_fwd_ws`` needs for these sizes on the current device."""
    Bt, L, H, P = x_shape
    d = make_dims(Bt, L, H, P, dstate, ngroups, chunk, dtype, path, schedule)
    n = ctypes.c_uint64(0)
    _check(_lib.ssd_scan_fwd_workspace_size(ctypes.byref(d), ctypes.byref(n)), "ssd_scan_fwd_workspace_size")
    return int(n.value)


def launch_count() -> int:
    return int(_lib.ssd_launch_count())


def device_error(stream=None) -> int:
    st = torch.cuda.current_stream() if stream is None else stream
    code = ctypes.c_uint32(0)
    _check(_lib.ssd_get_device_error(ctypes.c_void_p(st.cuda_stream), ctypes.byref(code)),
           "ssd_get_device_error")
    return int(code.value)


def ssd_scan_fwd(x, dt_raw, dt_bias, A_log, B, C, D, init_state=None, *, chunk=256,
                 path="auto", return_final_state=True, y=None, final_state=None, stream=None,
                 diag_stall_handoff=False, schedule="auto"):
    """Forward SSD scan on CUDA tensors.  Returns ``(y, final_state)``.

    ``x [B,L,H,P]`` and ``B, C [B,L,G,N]`` share one dtype (bf16 or fp32);
    ``dt_raw [B,L,H]``, ``dt_bias, A_log, D [H]`` and the states
    ``[B,H,P,N]`` are fp32.  Work is enqueued on ``stream`` (default: the
    current torch stream); the call does not synchronise.  ``schedule``
    requests the chunked path's schedule ("ranges", "pieces", "split"), or
    lets the library choose ("auto").
    """
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        Bt, L, H, P = x.shape
        final_state = torch.empty((Bt, H, P, B.shape[3]), dtype=torch.float32, device=x.device)
    for name, t in (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log),
                    ("B", B), ("C", C), ("D", D), ("init_state", init_state), ("y", y),
                    ("final_state", final_state)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    d = _dims_from(x, B, chunk, path, schedule)
    if diag_stall_handoff:
        d.flags |= DIAG_STALL_HANDOFF
    st = torch.cuda.current_stream(x.device) if stream is None else stream
    _check(_lib.ssd_scan_fwd(_ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A_log), _ptr(B), _ptr(C),
                             _ptr(D), _ptr(init_state), _ptr(y), _ptr(final_state),
                             ctypes.byref(d), ctypes.c_void_p(st.cuda_stream)),
           "ssd_scan_fwd")
    return y, final_state


def ssd_scan_fwd_host(x, dt_raw, dt_bias, A_log, B, C, D, init_state=None, *, chunk=256,
                      path="auto", return_final_state=True, y=None, final_state=None,
                      stream=None, device=None, schedule="auto"):
    """Same scan on CPU tensors (pinned for asynchronous copies).  The library
    copies in, runs, copies out and synchronises before returning."""
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        Bt, L, H, P = x.shape
        final_state = torch.empty((Bt, H, P, B.shape[3]), dtype=torch.float32)
    for name, t in (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log),
                    ("B", B), ("C", C), ("D", D), ("init_state", init_state), ("y", y),
                    ("final_state", final_state)):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    d = _dims_from(x, B, chunk, path, schedule)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        st = torch.cuda.current_stream(dev) if stream is None else stream
        _check(_lib.ssd_scan_fwd_host(_ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A_log), _ptr(B),
                                      _ptr(C), _ptr(D), _ptr(init_state), _ptr(y),
                                      _ptr(final_state), ctypes.byref(d),
                                      ctypes.c_void_p(st.cuda_stream)),
               "ssd_scan_fwd_host")
    return y, final_state


def ssd_scan_fwd_noalloc(x, dt_raw, dt_bias, A_log, B, C, D, init_state=None, *, chunk=256,
                         path="auto", y=None, final_state=None, return_final_state=True,
                         stream=None, schedule="auto"):
    """``ssd_scan_fwd`` on the chunked path with the library's fixed scratch
    array instead of a pool allocation (the library allocates nothing; outputs
    not passed in are created here by torch).  Calls that may overlap on one
    device share that array and race; calls ordered on one stream are safe."""
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        Bt, L, H, P = x.shape
        final_state = torch.empty((Bt, H, P, B.shape[3]), dtype=torch.float32, device=x.device)
    for name, t in (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log),
                    ("B", B), ("C", C), ("D", D), ("init_state", init_state), ("y", y),
                    ("final_state", final_state)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    d = _dims_from(x, B, chunk, path, schedule)
    st = torch.cuda.current_stream(x.device) if stream is None else stream
    _check(_lib.ssd_scan_fwd_noalloc(_ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A_log), _ptr(B),
                                     _ptr(C), _ptr(D), _ptr(init_state), _ptr(y),
                                     _ptr(final_state), ctypes.byref(d),
                                     ctypes.c_void_p(st.cuda_stream)),
           "ssd_scan_fwd_noalloc")
    return y, final_state


def ssd_scan_fwd_ws(x, dt_raw, dt_bias, A_log, B, C, D, init_state=None, *, workspace,
                    chunk=256, path="auto", y=None, final_state=None, return_final_state=True,
                    stream=None, schedule="auto"):
    """``ssd_scan_fwd`` with caller-provided scratch: ``workspace`` is a CUDA
    tensor of at least ``workspace_size(...)`` bytes (or None when that is 0).
    The library allocates nothing; calls that may overlap must not share a
    workspace."""
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        Bt, L, H, P = x.shape
        final_state = torch.empty((Bt, H, P, B.shape[3]), dtype=torch.float32, device=x.device)
    for name, t in (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log),
                    ("B", B), ("C", C), ("D", D), ("init_state", init_state), ("y", y),
                    ("final_state", final_state), ("workspace", workspace)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    d = _dims_from(x, B, chunk, path, schedule)
    st = torch.cuda.current_stream(x.device) if stream is None else stream
    _check(_lib.ssd_scan_fwd_ws(_ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A_log), _ptr(B), _ptr(C),
                                _ptr(D), _ptr(init_state), _ptr(y), _ptr(final_state),
                                _ptr(workspace), ctypes.c_uint64(nbytes), ctypes.byref(d),
                                ctypes.c_void_p(st.cuda_stream)),
           "ssd_scan_fwd_ws")
    return y, final_state


def ssd_trap_scan_fwd(v, k, q, dt, a, trap, D, h0=None, k0=None, v0=None, *, chunk=256, path="auto", y=None,
                      h_final=None, k_final=None, v_final=None, return_states=True, stream=None, schedule="auto"):
    """Trapezoidal (Mamba-3 SISO) scan on CUDA tensors.  Returns
    ``(y, h_final, k_final, v_final)`` (the states None when not returned).
    ``schedule`` requests a schedule of the chunked kernel, as for ``ssd_scan_fwd``.

    ``v [B,L,H,P]``, ``k, q [B,L,G,N]``, ``k0/k_final [B,H,N]`` and
    ``v0/v_final [B,H,P]`` share one dtype (bf16 or fp32); ``dt, a, trap
    [B,L,H]``, ``D [H]`` and ``h0/h_final [B,H,P,N]`` are fp32.
    """
    Bt, L, H, P = v.shape
    G, N = k.shape[2], k.shape[3]
    if y is None:
        y = torch.empty_like(v)
    if return_states:
        if h_final is None:
            h_final = torch.empty((Bt, H, P, N), dtype=torch.float32, device=v.device)
        if k_final is None:
            k_final = torch.empty((Bt, H, N), dtype=v.dtype, device=v.device)
        if v_final is None:
            v_final = torch.empty((Bt, H, P), dtype=v.dtype, device=v.device)
    named = (("v", v), ("k", k), ("q", q), ("dt", dt), ("a", a), ("trap", trap), ("D", D), ("h0", h0),
             ("k0", k0), ("v0", v0), ("y", y), ("h_final", h_final), ("k_final", k_final), ("v_final", v_final))
    for name, t in named:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    d = make_dims(Bt, L, H, P, N, G, chunk, v.dtype, path, schedule)
    st = torch.cuda.current_stream(v.device) if stream is None else stream
    _check(_lib.ssd_trap_scan_fwd(*(_ptr(t) for _, t in named), ctypes.byref(d),
                                  ctypes.c_void_p(st.cuda_stream)), "ssd_trap_scan_fwd")
    return y, h_final, k_final, v_final


def complex_scan_fwd(x, dt_raw, dt_bias, A_polar, B, C, D, init_state=None, *, path="auto", y=None,
                     final_state=None, return_state=True, stream=None):
    """Complex-valued scan with ET discretisation on CUDA tensors.  Returns
    ``(y, final_state)`` (the state None when not returned).

    ``x [B,L,H,P]`` and ``B, C [B,L,G,N]`` share one dtype (bf16 or fp32); B
    and C hold N/2 complex numbers as (re, im) pairs along N.  ``A_polar
    [H,2]`` = (log|A|, arg A), ``dt_raw [B,L,H]``, ``dt_bias, D [H]`` and the
    states ``[B,H,P,N]`` (complex as (re, im) pairs) are fp32.
    """
    Bt, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_state:
        final_state = torch.empty((Bt, H, P, N), dtype=torch.float32, device=x.device)
    named = (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_polar", A_polar), ("B", B), ("C", C),
             ("D", D), ("init_state", init_state), ("y", y), ("final_state", final_state))
    _require_cuda(named)
    d = make_dims(Bt, L, H, P, N, G, 1, x.dtype, path)
    st = torch.cuda.current_stream(x.device) if stream is None else stream
    _check(_lib.ssd_complex_scan_fwd(*(_ptr(t) for _, t in named), ctypes.byref(d),
                                     ctypes.c_void_p(st.cuda_stream)), "ssd_complex_scan_fwd")
    return y, final_state


def _require_cuda(named):
    for name, t in named:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")


def conv1d_silu_fwd(xbc, weight, bias=None, conv_state=None, *, nheads, headdim, ngroups, dstate,
                    x=None, B=None, C=None, conv_state_out=None, return_state=True, stream=None):
    """Causal depthwise conv1d + SiLU over the fused x | B | C channels of
    ``xbc [B,L,C]`` (``weight [C,K]``, ``bias [C]``, ``conv_state [B,K-1,C]``).
    Returns ``(x [B,L,H,P], B [B,L,G,N], C [B,L,G,N], conv_state_out)``."""
    Bt, L, Cc = xbc.shape
    K = weight.shape[1]
    if x is None:
        x = torch.empty((Bt, L, nheads, headdim), dtype=xbc.dtype, device=xbc.device)
    if B is None:
        B = torch.empty((Bt, L, ngroups, dstate), dtype=xbc.dtype, device=xbc.device)
    if C is None:
        C = torch.empty((Bt, L, ngroups, dstate), dtype=xbc.dtype, device=xbc.device)
    if conv_state_out is None and return_state:
        conv_state_out = torch.empty((Bt, K - 1, Cc), dtype=xbc.dtype, device=xbc.device)
    named = (("xbc", xbc), ("weight", weight), ("bias", bias), ("conv_state", conv_state), ("x", x),
             ("B", B), ("C", C), ("conv_state_out", conv_state_out))
    _require_cuda(named)
    d = make_dims(Bt, L, nheads, headdim, dstate, ngroups, 1, xbc.dtype)
    st = torch.cuda.current_stream(xbc.device) if stream is None else stream
    _check(_lib.ssd_conv1d_silu_fwd(*(_ptr(t) for _, t in named), ctypes.c_int32(K), ctypes.byref(d),
                                    ctypes.c_void_p(st.cuda_stream)), "ssd_conv1d_silu_fwd")
    return x, B, C, conv_state_out


def conv_scan_fwd(xbc, weight, bias, conv_state, dt_raw, dt_bias, A_log, D, init_state=None, *, nheads, headdim,
                  ngroups, dstate, chunk=256, y=None, final_state=None, conv_state_out=None, return_final_state=True,
                  return_conv_state=True, stream=None, path="auto", schedule="auto"):
    """``ssd_conv_scan_fwd``: the causal conv1d + SiLU over ``xbc [B,L,C]`` and the
    forward scan of its output, with the conv of the x channels inside the chunked
    scan kernel.  Returns ``(y [B,L,H,P], final_state, conv_state_out)``."""
    Bt, L, Cc = xbc.shape
    K = weight.shape[1]
    if y is None:
        y = torch.empty((Bt, L, nheads, headdim), dtype=xbc.dtype, device=xbc.device)
    if final_state is None and return_final_state:
        final_state = torch.empty((Bt, nheads, headdim, dstate), dtype=torch.float32, device=xbc.device)
    if conv_state_out is None and return_conv_state:
        conv_state_out = torch.empty((Bt, K - 1, Cc), dtype=xbc.dtype, device=xbc.device)
    named = (("xbc", xbc), ("weight", weight), ("bias", bias), ("conv_state", conv_state))
    rest = (("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log), ("D", D), ("init_state", init_state),
            ("y", y), ("final_state", final_state), ("conv_state_out", conv_state_out))
    _require_cuda(named + rest)
    d = make_dims(Bt, L, nheads, headdim, dstate, ngroups, chunk, xbc.dtype, path, schedule)
    st = torch.cuda.current_stream(xbc.device) if stream is None else stream
    _check(_lib.ssd_conv_scan_fwd(*(_ptr(t) for _, t in named), ctypes.c_int32(K), *(_ptr(t) for _, t in rest),
                                  ctypes.byref(d), ctypes.c_void_p(st.cuda_stream)), "ssd_conv_scan_fwd")
    return y, final_state, conv_state_out


def gated_rmsnorm_fwd(y, z, weight, eps=1e-6, *, out=None, stream=None):
    """RMSNorm(y) * weight * SiLU(z) per token over the H*P channels of
    ``y, z [B,L,H,P]`` (``weight [H*P]`` fp32)."""
    Bt, L, H, P = y.shape
    if out is None:
        out = torch.empty_like(y)
    named = (("y", y), ("z", z), ("weight", weight), ("out", out))
    _require_cuda(named)
    d = make_dims(Bt, L, H, P, 1, 1, 1, y.dtype)
    st = torch.cuda.current_stream(y.device) if stream is None else stream
    _check(_lib.ssd_gated_rmsnorm_fwd(_ptr(y), _ptr(z), _ptr(weight), ctypes.c_float(eps), _ptr(out),
                                      ctypes.byref(d), ctypes.c_void_p(st.cuda_stream)), "ssd_gated_rmsnorm_fwd")
    return out


def ssd_scan_bwd(x, dt_raw, dt_bias, A_log, B, C, D, init_state, dy, d_final=None, *, path="auto",
                 stream=None, fp32_form=False, split_states=False):
    """Gradients of ``ssd_scan_fwd`` given ``dy`` (and ``d_final``).  Returns a
    dict of fp32 CUDA tensors: dx, ddt_raw, ddt_bias, dA_log, dB, dC, dD, d_init.
    ``fp32_form`` keeps the chunk form's fp32 contractions where its tensor-core
    form would apply (bf16, P = 64, N = 128); ``split_states`` computes that
    form's chunk states and chains in two launches instead of one walk."""
    Bt, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    f32 = dict(dtype=torch.float32, device=x.device)
    out = dict(dx=torch.empty((Bt, L, H, P), **f32), ddt_raw=torch.empty((Bt, L, H), **f32),
               ddt_bias=torch.empty((H,), **f32), dA_log=torch.empty((H,), **f32),
               dB=torch.empty((Bt, L, G, N), **f32), dC=torch.empty((Bt, L, G, N), **f32),
               dD=torch.empty((H,), **f32), d_init=torch.empty((Bt, H, P, N), **f32))
    named = (("x", x), ("dt_raw", dt_raw), ("dt_bias", dt_bias), ("A_log", A_log), ("B", B), ("C", C), ("D", D),
             ("init_state", init_state), ("dy", dy), ("d_final", d_final)) + tuple(out.items())
    _require_cuda(named)
    d = make_dims(Bt, L, H, P, N, G, 1, x.dtype, path)
    if fp32_form:
        d.flags |= BWD_FP32_FORM
    if split_states:
        d.flags |= BWD_SPLIT_STATES
    st = torch.cuda.current_stream(x.device) if stream is None else stream
    _check(_lib.ssd_scan_bwd(*(_ptr(t) for _, t in named), ctypes.byref(d), ctypes.c_void_p(st.cuda_stream)),
           "ssd_scan_bwd")
    return out


# ---- the attention layers of hybrid stacks: a step's plan, queries and keys, attention over the paged cache ----
# Tensors, stream and workspace of a call are of the thread's current device (else ValueError).

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream_ptr(device, stream):
    """The stream's handle.  The library works on the thread's current device, so that has to be the tensors', and the
    stream's: checked on every call."""
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device_index != device.index:
        raise ValueError(f"the tensors are on {device}, the stream is not")
    return stream.cuda_stream


def _layout(t):
    """What the checks of an argument go by: everything but its address."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


# Call structures of argument layouts that have passed the checks below: a serving loop calls with the same few
# layouts again and again, and the checks and the structure cost several times the call itself.  Nothing of an
# argument's address or contents is kept.
_known = {}


def _remember(key, d):
    if len(_known) >= 4096:
        _known.clear()
    _known[key] = d
    return d


def _vectors(device, named, dtype):
    """Contiguous 1-d tensors of ``dtype`` on ``device`` (``named``: (name, tensor or None, length or None))."""
    for name, t, n in named:
        if t is None:
            continue
        if t.dtype != dtype or t.device != device or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-d {dtype} tensor on {device}")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements, not {t.shape[0]}")


def _rows(device, named, dtype):
    """[n, heads, D] tensors of ``dtype`` with a contiguous last axis (``named``: (name, tensor or None, shape))."""
    for name, t, shape in named:
        if t is None:
            continue
        if t.dtype != dtype or t.device != device or t.shape != shape:
            raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on {device}")
        if t.stride(2) != 1 and shape[2] != 1:
            raise ValueError(f"{name} must have a contiguous last axis")


def _cache_args(device, dtype, k_cache, v_cache, heads, D):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[2] != heads or k_cache.shape[3] != D:
        raise ValueError(f"k_cache and v_cache must be [npages, page_size, {heads}, {D}]")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != dtype or t.device != device or t.stride(3) != 1:
            raise ValueError(f"{name} must be a {dtype} tensor on {device} with a contiguous last axis")


def _workspace(workspace, device):
    if workspace is None:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def paged_plan(lens, new_lens, block_table, free_ring, ring_pos, *, page_size, max_tokens, out=None, stream=None):
    """Block tables, positions and slots of one serving step, on the GPU (``ssd_paged_plan``).

    ``lens, new_lens [R]`` int32: tokens each request holds, and brings (negative: finished, its pages go back);
    ``block_table [R, max_pages]`` int32 and ``free_ring [n]`` int32 are updated in place; ``ring_pos [2]`` int64 is
    the ring's head and tail.  Returns a dict of ``lens, granted [R]``, ``start [R+1]``, ``positions, token_req,
    slots [max_tokens]`` (-1 past ``start[R]``), ``ring_pos [2]`` and ``counts [4]`` (tokens granted, pages taken,
    pages given back, requests refused); slots and ring_pos int64, the others int32.  ``out`` gives the tensors to
    write, as such a dict; its ``lens`` and ``ring_pos`` may be the inputs (in place).
    """
    R, dev = lens.shape[0], lens.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        i64 = dict(dtype=torch.int64, device=dev)
        out = dict(lens=torch.empty(R, **i32), granted=torch.empty(R, **i32), start=torch.empty(R + 1, **i32),
                   positions=torch.empty(max_tokens, **i32), token_req=torch.empty(max_tokens, **i32),
                   slots=torch.empty(max_tokens, **i64), ring_pos=torch.empty(2, **i64), counts=torch.empty(4, **i32))
    o = out
    key = (paged_plan, *map(_layout, (lens, new_lens, block_table, free_ring, ring_pos, o["lens"], o["granted"], o["start"],
                                      o["positions"], o["token_req"], o["slots"], o["ring_pos"], o["counts"])), page_size, max_tokens)
    d = _known.get(key)
    if d is None:
        if not lens.is_cuda:
            raise ValueError("lens must be a CUDA tensor")
        if block_table.dtype != torch.int32 or block_table.device != dev or block_table.dim() != 2 or \
                block_table.shape[0] != R or not block_table.is_contiguous():
            raise ValueError(f"block_table must be a contiguous [{R}, max_pages] int32 tensor on {dev}")
        _vectors(dev, (("lens", lens, R), ("new_lens", new_lens, R), ("free_ring", free_ring, None), ("out lens", o["lens"], R),
                       ("granted", o["granted"], R), ("start", o["start"], R + 1), ("positions", o["positions"], max_tokens),
                       ("token_req", o["token_req"], max_tokens), ("counts", o["counts"], 4)), torch.int32)
        _vectors(dev, (("ring_pos", ring_pos, 2), ("out ring_pos", o["ring_pos"], 2), ("slots", o["slots"], max_tokens)),
                 torch.int64)
        d = _remember(key, SsdPlanDims(R, max_tokens, free_ring.shape[0], page_size, block_table.shape[1], 0, 0))
    st = _stream_ptr(dev, stream)
    _check(_lib.ssd_paged_plan(lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), free_ring.data_ptr(),
                               ring_pos.data_ptr(), o["lens"].data_ptr(), o["granted"].data_ptr(), o["start"].data_ptr(),
                               o["positions"].data_ptr(), o["token_req"].data_ptr(), o["slots"].data_ptr(),
                               o["ring_pos"].data_ptr(), o["counts"].data_ptr(), d, st),
           "ssd_paged_plan")
    return out


def rope_table(max_pos, rotary_dim, base=10000.0, device="cuda"):
    """``(cos, sin)``, each ``[max_pos, rotary_dim / 2]`` fp32, of the angles ``pos * base^(-2 i / rotary_dim)``,
    computed in fp64."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * base ** (-2.0 * i / max(rotary_dim, 1))[None, :]
    return ang.cos().float().to(device), ang.sin().float().to(device)


def _qk_dims(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a [tokens, heads, D] CUDA tensor")
    T, Hq, D = q.shape
    dev = q.device
    if q.dtype not in _DTYPES:
        raise SsdError(9, "q must be bf16 or fp32")
    if k.dim() != 3:
        raise ValueError("k must be a [tokens, heads, D] CUDA tensor")
    Hk = k.shape[1]
    _rows(dev, (("q", q, (T, Hq, D)), ("k", k, (T, Hk, D))), q.dtype)
    _vectors(dev, (("q_weight", q_weight, D), ("k_weight", k_weight, D)), torch.float32)
    _vectors(dev, (("positions", positions, T),), torch.int32)
    for name, t in (("cos", cos), ("sin", sin)):
        if t.dtype != torch.float32 or t.device != dev or t.dim() != 2 or t.shape != cos.shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [max_pos, rotary_dim / 2] fp32 tensor on {dev}, as the other is")
    d = SsdQkDims(T, cos.shape[0], 0, Hq, Hk, D, 2 * cos.shape[1], 0, _DTYPES[q.dtype],
                  ROPE_INTERLEAVED if interleaved else 0, eps, q.stride()[:2], k.stride()[:2])
    return d


def qk_norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions, *, eps=1e-6, interleaved=False, v=None, k_cache=None,
                     v_cache=None, slots=None, q_out=None, k_out=None, return_k=True, stream=None):
    """RMSNorm of every query and key head and the rotary position in one pass (``ssd_qk_norm_rope_fwd``).
    Returns ``(q_out, k_out)``.

    ``q [T,Hq,D]`` and ``k, v [T,Hk,D]`` in bf16 or fp32 with a contiguous last axis (views of a fused projection are
    fine); ``q_weight, k_weight [D]`` fp32 or None; ``cos, sin [max_pos, R/2]`` fp32 (:func:`rope_table`);
    ``positions [T]`` int32 (a token whose position is outside the table is padding).  Given ``v``, ``k_cache, v_cache
    [npages, page_size, Hk, D]`` (any strides, contiguous last axis) and ``slots [T]`` int64, keys and values go into
    the cache as well; ``return_k=False`` then leaves ``k_out`` out (None).  ``q_out`` may be ``q`` and ``k_out`` ``k``.
    """
    dev = q.device
    key = (qk_norm_rope_fwd, *map(_layout, (q, k, q_weight, k_weight, cos, sin, positions, v, k_cache, v_cache, slots, q_out,
                                            k_out)), eps, interleaved, return_k)
    d = _known.get(key)
    if d is None:   # (first of all, so that only tensors that are CUDA tensors get outputs)
        d = _qk_dims(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        _rows(dev, (("q_out", q_out, q.shape), ("k_out", k_out, k.shape), ("v", v, k.shape)), q.dtype)
        d.qo_stride = (q.shape[1] * q.shape[2], q.shape[2]) if q_out is None else q_out.stride()[:2]
        d.ko_stride = (k.shape[1] * k.shape[2], k.shape[2]) if k_out is None else k_out.stride()[:2]
        if k_cache is not None or v_cache is not None or slots is not None:
            if k_cache is None or v_cache is None or slots is None or v is None:
                raise ValueError("writing the cache takes v, k_cache, v_cache and slots")
            _cache_args(dev, q.dtype, k_cache, v_cache, k.shape[1], q.shape[2])
            _vectors(dev, (("slots", slots, q.shape[0]),), torch.int64)
            d.npages, d.page_size = k_cache.shape[0], k_cache.shape[1]
            d.v_stride, d.kc_stride, d.vc_stride = v.stride()[:2], k_cache.stride()[:3], v_cache.stride()[:3]
        elif k_out is None and not return_k:
            raise ValueError("return_k=False takes a cache to write the keys to")
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if k_out is None and return_k:
        k_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
    _check(_lib.ssd_qk_norm_rope_fwd(q.data_ptr(), k.data_ptr(), _addr(v), _addr(q_weight), _addr(k_weight), cos.data_ptr(),
                                     sin.data_ptr(), positions.data_ptr(), q_out.data_ptr(), _addr(k_out), _addr(k_cache),
                                     _addr(v_cache), _addr(slots), d, st), "ssd_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, *, eps=1e-6, interleaved=False, dq=None,
                     dk=None, workspace=None, stream=None):
    """Gradients of :func:`qk_norm_rope_fwd` given those of its outputs.  Returns a dict: ``dq, dk`` in the inputs'
    dtype, ``dq_weight, dk_weight [D]`` fp32.  ``dq`` and ``dk`` may be given (views of a fused gradient, or ``dq_out``
    and ``dk_out`` themselves)."""
    dev, D = q.device, q.shape[2]
    key = (qk_norm_rope_bwd, *map(_layout, (q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk)), eps,
           interleaved)
    d = _known.get(key)
    if d is None:
        d = _qk_dims(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        _rows(dev, (("dq_out", dq_out, q.shape), ("dk_out", dk_out, k.shape), ("dq", dq, q.shape), ("dk", dk, k.shape)), q.dtype)
        d.qo_stride, d.ko_stride = dq_out.stride()[:2], dk_out.stride()[:2]
        d.dq_stride = (q.shape[1] * D, D) if dq is None else dq.stride()[:2]
        d.dk_stride = (k.shape[1] * D, D) if dk is None else dk.stride()[:2]
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if dq is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if dk is None:
        dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
    dqw, dkw = torch.empty(D, dtype=torch.float32, device=dev), torch.empty(D, dtype=torch.float32, device=dev)
    ws, nws = _workspace(workspace, dev)
    _check(_lib.ssd_qk_norm_rope_bwd(q.data_ptr(), k.data_ptr(), _addr(q_weight), _addr(k_weight), cos.data_ptr(),
                                     sin.data_ptr(), positions.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(),
                                     dq.data_ptr(), dk.data_ptr(), dqw.data_ptr(), dkw.data_ptr(), ws, nws, d, st),
           "ssd_qk_norm_rope_bwd")
    return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)


def qk_norm_rope_bwd_workspace_size(q, k) -> int:
    """Bytes of scratch ``qk_norm_rope_bwd`` needs for such tensors on the current device."""
    d = SsdQkDims(q.shape[0], 0, 0, q.shape[1], k.shape[1], q.shape[2], 0, 0, _DTYPES[q.dtype], 0, 0.0)
    n = ctypes.c_uint64(0)
    _check(_lib.ssd_qk_norm_rope_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)), "ssd_qk_norm_rope_bwd_workspace_size")
    return int(n.value)


def _attn_dims(q, k_cache, v_cache, block_table, scale, window):
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a [rows, heads, D] CUDA tensor")
    if q.dtype not in _DTYPES:
        raise SsdError(9, "q must be bf16 or fp32")
    n, H, D = q.shape
    dev = q.device
    _rows(dev, (("q", q, (n, H, D)),), q.dtype)
    _cache_args(dev, q.dtype, k_cache, v_cache, k_cache.shape[2], D)
    if block_table.dtype != torch.int32 or block_table.device != dev or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table must be a [requests, max_pages] int32 tensor on {dev} with contiguous rows")
    return SsdAttnDims(n, block_table.shape[0], k_cache.shape[0], H, k_cache.shape[2], D, k_cache.shape[1],
                       block_table.shape[1], window, _DTYPES[q.dtype], 0, D ** -0.5 if scale is None else scale, 0,
                       q.stride()[:2], q.stride()[:2], k_cache.stride()[:3], v_cache.stride()[:3], block_table.stride(0))


def paged_attn_fwd(q, k_cache, v_cache, block_table, positions, start=None, *, scale=None, window=0, out=None, lse=None,
                   return_lse=True, workspace=None, stream=None):
    """Attention of new tokens over a paged key-value cache (``ssd_paged_attn_fwd``).  Returns ``(out, lse)``.

    ``q [rows,H,D]``; ``k_cache, v_cache [npages, page_size, Hkv, D]`` (any strides, contiguous last axis; H a multiple
    of Hkv); ``block_table [R, max_pages]`` int32; ``positions [rows]`` int32: each row sees its request's cached
    positions up to its own (the last ``window`` of them, if given).  Without ``start`` row i is request i's one new
    token; with ``start [R+1]`` int32 request r has the rows ``start[r] .. start[r+1]-1``, as :func:`paged_plan` gives
    them.  Rows that see nothing get 0 (lse -inf).  ``scale`` defaults to D^-1/2.  ``out [rows,H,D]`` is in q's dtype,
    ``lse [rows,H]`` fp32.
    """
    dev = q.device
    key = (paged_attn_fwd, *map(_layout, (q, k_cache, v_cache, block_table, positions, start, out, lse)), scale, window)
    d = _known.get(key)
    if d is None:
        d = _attn_dims(q, k_cache, v_cache, block_table, scale, window)
        n, H, D = q.shape
        _rows(dev, (("out", out, q.shape),), q.dtype)
        if lse is not None and (lse.dtype != torch.float32 or lse.device != dev or lse.shape != (n, H) or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous [{n}, {H}] fp32 tensor on {dev}")
        _vectors(dev, (("positions", positions, n), ("start", start, block_table.shape[0] + 1)), torch.int32)
        d.o_stride = (H * D, D) if out is None else out.stride()[:2]
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if lse is None and return_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    ws, nws = _workspace(workspace, dev)
    _check(_lib.ssd_paged_attn_fwd(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                   positions.data_ptr(), _addr(start), out.data_ptr(), _addr(lse), ws, nws, d, st),
           "ssd_paged_attn_fwd")
    return out, lse


def paged_attn_workspace_size(q, k_cache, v_cache, block_table) -> int:
    """Bytes of scratch ``paged_attn_fwd`` needs for such tensors on the current device."""
    d = _attn_dims(q, k_cache, v_cache, block_table, 1.0, 0)
    n = ctypes.c_uint64(0)
    _check(_lib.ssd_paged_attn_workspace_size(ctypes.byref(d), ctypes.byref(n)), "ssd_paged_attn_workspace_size")
    return int(n.value)


# ---- one layer's step around the scan: residual norm, 8-bit products, conv and scan for single tokens ----
# Devices, streams and workspaces as for the attention layers' calls.

def _matrix(device, named):
    """[n, width] tensors with a contiguous last axis (``named``: (name, tensor or None, dtype, shape))."""
    for name, t, dtype, shape in named:
        if t is None:
            continue
        if t.dtype != dtype or t.device != device or t.shape != shape:
            raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on {device}")
        if shape[1] != 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have a contiguous last axis")


def _contiguous(device, named):
    """Contiguous tensors (``named``: (name, tensor or None, dtype, shape))."""
    for name, t, dtype, shape in named:
        if t is None:
            continue
        if t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")


def _norm_dims(x, name, weight, residual_dtype, eps):
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a [rows, D] CUDA tensor")
    if x.dtype not in _DTYPES or residual_dtype not in _DTYPES:
        raise SsdError(9, f"{name} and the residual must be bf16 or fp32")
    n, D = x.shape
    _matrix(x.device, ((name, x, x.dtype, x.shape),))
    _vectors(x.device, (("weight", weight, D),), torch.float32)
    return SsdNormDims(n, D, _DTYPES[x.dtype], _DTYPES[residual_dtype], 0, eps, 0, x.stride(0), 0, 0, D, D, D)


def _add_rmsnorm(what, x, weight, residual, eps, out, q, scale, residual_out, return_residual, stream):
    dev = x.device
    key = (what, *map(_layout, (x, weight, residual, out, q, scale, residual_out)), eps, return_residual)
    d = _known.get(key)
    if d is None:
        d = _norm_dims(x, "x", weight, x.dtype if residual is None else residual.dtype, eps)
        if residual is None and residual_out is not None:
            raise ValueError("residual_out without a residual")
        for name, t, dtype in (("residual", residual, residual.dtype if residual is not None else None), ("out", out, x.dtype),
                               ("q", q, torch.int8), ("residual_out", residual_out, residual.dtype if residual is not None else None)):
            _matrix(dev, ((name, t, dtype, x.shape),))
        _vectors(dev, (("scale", scale, x.shape[0]),), torch.float32)
        for field, t in (("residual_stride", residual), ("out_stride", out), ("ro_stride", residual_out), ("q_stride", q)):
            if t is not None:
                setattr(d, field, t.stride(0))
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if what is add_rmsnorm_fwd:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        if q is None:
            q = torch.empty(x.shape, dtype=torch.int8, device=dev)
        if scale is None:
            scale = torch.empty(x.shape[0], dtype=torch.float32, device=dev)
    if residual is not None and residual_out is None and return_residual:
        residual_out = torch.empty(x.shape, dtype=residual.dtype, device=dev)
    _check(_lib.ssd_add_rmsnorm_fwd(x.data_ptr(), _addr(residual), weight.data_ptr(), _addr(out), _addr(q), _addr(scale),
                                    _addr(residual_out), d, st), "ssd_add_rmsnorm_fwd")
    return out, q, scale, residual_out


def add_rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, out=None, residual_out=None, return_residual=True, stream=None):
    """``h = x + residual`` and ``out = h / sqrt(mean(h^2) + eps) * weight`` per row (``ssd_add_rmsnorm_fwd``).
    Returns ``(out, residual_out)``.

    ``x [rows, D]`` in bf16 or fp32, ``residual`` in x's dtype or fp32 (None: h is x and nothing is returned for it),
    ``weight [D]`` fp32; rows may have any stride of whole 16 bytes.  ``residual_out`` (h, in the residual's dtype) may
    be ``residual`` and ``out`` may be ``x``; ``return_residual=False`` leaves h out (None)."""
    out, _, _, residual_out = _add_rmsnorm(add_rmsnorm_fwd, x, weight, residual, eps, out, None, None, residual_out, return_residual, stream)
    return out, residual_out


def add_rmsnorm_q8_fwd(x, weight, residual=None, *, eps=1e-6, q=None, scale=None, residual_out=None, return_residual=True,
                       stream=None):
    """:func:`add_rmsnorm_fwd` with an 8-bit result: ``q [rows, D]`` int8 and ``scale [rows]`` fp32, standing for
    ``q * scale[:, None]``.  Returns ``(q, scale, residual_out)``."""
    _, q, scale, residual_out = _add_rmsnorm(add_rmsnorm_q8_fwd, x, weight, residual, eps, None, q, scale, residual_out, return_residual,
                                             stream)
    return q, scale, residual_out


def gated_rmsnorm_q8_fwd(y, z, weight, eps=1e-6, *, q=None, scale=None, stream=None):
    """``RMSNorm(y) * weight * SiLU(z)`` per row (:func:`gated_rmsnorm_fwd`) with an 8-bit result, as
    :func:`add_rmsnorm_q8_fwd` gives it (``ssd_gated_rmsnorm_q8_fwd``).  ``y, z [rows, D]``, z at any row stride (a slice of the projection).  Returns
    ``(q, scale)``."""
    dev = y.device
    key = (gated_rmsnorm_q8_fwd, *map(_layout, (y, z, weight, q, scale)), eps)
    d = _known.get(key)
    if d is None:
        d = _norm_dims(y, "y", weight, y.dtype, eps)
        _matrix(dev, (("z", z, y.dtype, y.shape), ("q", q, torch.int8, y.shape)))
        _vectors(dev, (("scale", scale, y.shape[0]),), torch.float32)
        d.z_stride = z.stride(0)
        d.q_stride = y.shape[1] if q is None else q.stride(0)
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if q is None:
        q = torch.empty(y.shape, dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(y.shape[0], dtype=torch.float32, device=dev)
    _check(_lib.ssd_gated_rmsnorm_q8_fwd(y.data_ptr(), z.data_ptr(), weight.data_ptr(), q.data_ptr(), scale.data_ptr(), d, st),
           "ssd_gated_rmsnorm_q8_fwd")
    return q, scale


def add_rmsnorm_bwd(h, weight, dout, dresidual=None, *, eps=1e-6, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of :func:`add_rmsnorm_fwd` (``ssd_add_rmsnorm_bwd``).  ``h`` is its ``residual_out`` (without a residual:
    x), ``dout`` and ``dresidual`` the gradients of its outputs.  Returns ``(dx, dweight)``: the gradient of x and of the
    residual alike, in h's dtype, and that of the weight in fp32.  ``dx`` may be ``dresidual``, or ``dout`` where that
    is in h's dtype."""
    dev = h.device
    key = (add_rmsnorm_bwd, *map(_layout, (h, weight, dout, dresidual, dx, dweight)), eps)
    d = _known.get(key)
    if d is None:
        d = _norm_dims(dout, "dout", weight, h.dtype, eps)
        _matrix(dev, (("h", h, h.dtype, dout.shape), ("dout", dout, dout.dtype, dout.shape), ("dresidual", dresidual, h.dtype, dout.shape),
                      ("dx", dx, h.dtype, dout.shape)))
        _vectors(dev, (("dweight", dweight, h.shape[1]),), torch.float32)
        d.ro_stride = h.stride(0)
        for field, t in (("residual_stride", dresidual), ("out_stride", dx)):
            if t is not None:
                setattr(d, field, t.stride(0))
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if dx is None:
        dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    if dweight is None:
        dweight = torch.empty(h.shape[1], dtype=torch.float32, device=dev)
    ws, nws = _workspace(workspace, dev)
    _check(_lib.ssd_add_rmsnorm_bwd(h.data_ptr(), weight.data_ptr(), dout.data_ptr(), _addr(dresidual), dx.data_ptr(), dweight.data_ptr(),
                                    ws, nws, d, st), "ssd_add_rmsnorm_bwd")
    return dx, dweight


def add_rmsnorm_bwd_workspace_size(h, dout) -> int:
    """Bytes of scratch ``add_rmsnorm_bwd`` needs for such tensors on the current device."""
    d = SsdNormDims(h.shape[0], h.shape[1], _DTYPES[dout.dtype], _DTYPES[h.dtype])
    n = ctypes.c_uint64(0)
    _check(_lib.ssd_add_rmsnorm_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)), "ssd_add_rmsnorm_bwd_workspace_size")
    return int(n.value)


def q8_pack_weight(w, *, packed=None, stream=None):
    """``w [N, K]`` int8 in the order in which :func:`q8_matmul` reads it (``ssd_q8_pack_weight``): once per weight."""
    if w.dim() != 2 or not w.is_cuda:
        raise ValueError("w must be a [N, K] CUDA tensor")
    N, K = w.shape
    _matrix(w.device, (("w", w, torch.int8, w.shape),))
    size = -(-N // 128) * 128 * (-(-K // 64) * 64)
    _vectors(w.device, (("packed", packed, size),), torch.int8)
    st = _stream_ptr(w.device, stream)
    if packed is None:
        packed = torch.empty(size, dtype=torch.int8, device=w.device)
    _check(_lib.ssd_q8_pack_weight(w.data_ptr(), packed.data_ptr(), SsdQ8Dims(0, N, K, 0, 0, w.stride(0), N), st), "ssd_q8_pack_weight")
    return packed


def _q8_dims(a, N, dtype):
    if a.dim() != 2 or not a.is_cuda:
        raise ValueError("a must be a [tokens, K] CUDA tensor")
    if dtype not in _DTYPES:
        raise SsdError(9, "the result must be bf16 or fp32")
    _matrix(a.device, (("a", a, torch.int8, a.shape),))
    return SsdQ8Dims(a.shape[0], N, a.shape[1], _DTYPES[dtype], 0, a.stride(0), N)


def q8_matmul(a, a_scale, packed, w_scale, *, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """Products of 8-bit integers with a scale per token and per output channel (``ssd_q8_matmul``):
    ``(a @ w.T) * a_scale[:, None] * w_scale`` with the sums exact.  Returns ``[tokens, N]`` in ``dtype`` (bf16 or fp32; that
    of ``out``, if given).

    ``a [tokens, K]`` int8 (any row stride) and ``a_scale [tokens]`` as the norms give them; ``packed`` from
    :func:`q8_pack_weight`, ``w_scale [N]`` fp32."""
    dev = a.device
    if out is not None:
        dtype = out.dtype
    key = (q8_matmul, *map(_layout, (a, a_scale, packed, w_scale, out)), dtype)
    d = _known.get(key)
    if d is None:
        N = w_scale.shape[0]
        d = _q8_dims(a, N, dtype)
        _vectors(dev, (("a_scale", a_scale, a.shape[0]), ("w_scale", w_scale, N)), torch.float32)
        _vectors(dev, (("packed", packed, -(-N // 128) * 128 * (-(-a.shape[1] // 64) * 64)),), torch.int8)
        _matrix(dev, (("out", out, dtype, (a.shape[0], N)),))
        if out is not None:
            d.y_stride = out.stride(0)
        _remember(key, d)
    st = _stream_ptr(dev, stream)
    if out is None:
        out = torch.empty((a.shape[0], w_scale.shape[0]), dtype=dtype, device=dev)
    ws, nws = _workspace(workspace, dev)
    _check(_lib.ssd_q8_matmul(a.data_ptr(), a_scale.data_ptr(), packed.data_ptr(), w_scale.data_ptr(), out.data_ptr(), ws, nws, d, st),
           "ssd_q8_matmul")
    return out


def q8_matmul_workspace_size(a, N) -> int:
    """Bytes of scratch ``q8_matmul`` needs for such tokens and N output channels on the current device."""
    n = ctypes.c_uint64(0)
    _check(_lib.ssd_q8_matmul_workspace_size(ctypes.byref(_q8_dims(a, N, torch.float32)), ctypes.byref(n)), "ssd_q8_matmul_workspace_size")
    return int(n.value)


def conv_scan_step(xbc, conv_ring, weight, bias, dt_raw, dt_bias, A_log, D, states, slots, positions, *, ngroups, y=None,
                   stream=None):
    """The causal conv1d + SiLU and the scan (:func:`conv_scan_fwd`) for one token of each of several sequences, on a
    pool of their states (``ssd_conv_scan_step``).  Returns ``y [rows, H, P]``.

    Row i is the token at ``positions[i]`` of the sequence in ``slots[i]`` (both int32); a slot outside the pool or a
    negative position makes it padding (y zero, nothing else written).  ``conv_ring [nslots, K, C]`` (xbc's dtype; the input
    of position p in entry p mod K, see :func:`conv_ring_store`) and ``states [nslots, H, P, N]`` fp32 are updated in place;
    at position 0 neither is read.  ``xbc [rows, C]`` and ``dt_raw [rows, H]`` (xbc's dtype or fp32) may be views of one
    projection; ``weight [C, K]``, ``bias [C]`` or None, ``dt_bias, A_log, D [H]`` fp32."""
    dev = xbc.device
    key = (conv_scan_step, *map(_layout, (xbc, conv_ring, weight, bias, dt_raw, dt_bias, A_log, D, states, slots, positions, y)), ngroups)
    d = _known.get(key)
    if d is None:
        if xbc.dim() != 2 or not xbc.is_cuda:
            raise ValueError("xbc must be a [rows, C] CUDA tensor")
        if xbc.dtype not in _DTYPES or dt_raw.dtype not in _DTYPES:
            raise SsdError(9, "xbc and dt_raw must be bf16 or fp32")
        if states.dim() != 4 or weight.dim() != 2:
            raise ValueError("states must be [nslots, H, P, N] and weight [C, K]")
        n, C = xbc.shape
        S, H, P, N = states.shape
        K = weight.shape[1]
        if C != H * P + 2 * ngroups * N:
            raise ValueError(f"xbc must have H P + 2 G N = {H * P + 2 * ngroups * N} channels")
        _matrix(dev, (("xbc", xbc, xbc.dtype, (n, C)), ("dt_raw", dt_raw, dt_raw.dtype, (n, H))))
        _contiguous(dev, (("conv_ring", conv_ring, xbc.dtype, (S, K, C)), ("weight", weight, torch.float32, (C, K)),
                          ("states", states, torch.float32, (S, H, P, N))))
        _vectors(dev, (("bias", bias, C), ("dt_bias", dt_bias, H), ("A_log", A_log, H), ("D", D, H)), torch.float32)
        _vectors(dev, (("slots", slots, n), ("positions", positions, n)), torch.int32)
        if y is not None and (y.dtype != xbc.dtype or y.device != dev or y.shape != (n, H, P) or
                              (P > 1 and y.stride(2) != 1) or (H > 1 and y.stride(1) != P)):
            raise ValueError(f"y must be a {(n, H, P)} {xbc.dtype} tensor on {dev} with contiguous rows")
        d = _remember(key, SsdStepDims(n, S, H, P, N, ngroups, K, _DTYPES[xbc.dtype], _DTYPES[dt_raw.dtype], 0, xbc.stride(0),
                                       dt_raw.stride(0), H * P if y is None else y.stride(0)))
    st = _stream_ptr(dev, stream)
    if y is None:
        y = torch.empty((xbc.shape[0], *states.shape[1:3]), dtype=xbc.dtype, device=dev)
    _check(_lib.ssd_conv_scan_step(xbc.data_ptr(), conv_ring.data_ptr(), weight.data_ptr(), _addr(bias), dt_raw.data_ptr(),
                                   dt_bias.data_ptr(), A_log.data_ptr(), D.data_ptr(), states.data_ptr(), slots.data_ptr(),
                                   positions.data_ptr(), y.data_ptr(), d, st), "ssd_conv_scan_step")
    return y


def conv_ring_store(conv_ring, conv_state, slots, lengths, *, stream=None):
    """Puts a prompt's carried inputs where :func:`conv_scan_step` looks for them: ``conv_state [B, K-1, C]`` as
    :func:`conv1d_silu_fwd` or :func:`conv_scan_fwd` returns it, of sequences that now hold ``lengths [B]`` tokens, into the
    entries of ``slots [B]`` in ``conv_ring [nslots, K, C]`` (slots and lengths int32 or int64).  As there, a slot outside
    the pool or a negative length makes a row padding, and two rows must not have the same slot."""
    dev = conv_ring.device
    if conv_ring.dim() != 3 or conv_ring.shape[1] < 2 or conv_ring.dtype not in _DTYPES:
        raise ValueError("conv_ring must be a [nslots, K, C] bf16 or fp32 tensor")
    S, K, C = conv_ring.shape
    for name, t in (("slots", slots), ("lengths", lengths)):
        if t.dim() != 1 or t.shape != slots.shape or t.dtype not in (torch.int32, torch.int64) or t.device != dev:
            raise ValueError(f"{name} must be a [B] int32 or int64 tensor on {dev}")
    B = slots.shape[0]
    if conv_state.shape != (B, K - 1, C) or conv_state.dtype != conv_ring.dtype or conv_state.device != dev:
        raise ValueError(f"conv_state must be a {(B, K - 1, C)} {conv_ring.dtype} tensor on {dev}")
    if conv_ring.is_cuda:
        _stream_ptr(dev, stream)
    if S == 0 or B == 0:
        return
    with torch.cuda.stream(stream):
        slots, lengths = slots.long(), lengths.long()
        real = (slots >= 0) & (slots < S) & (lengths >= 0)
        # Padding stores what another row stores, in the same place; where all rows are padding, what is there.
        row = torch.where(real, torch.arange(B, device=dev), real.byte().argmax())
        to = slots[row].clamp(0, S - 1)[:, None]
        at = (lengths[row][:, None] - (K - 1) + torch.arange(K - 1, device=dev)) % K
        conv_ring[to, at] = torch.where(real.any(), conv_state[row], conv_ring[to, at])
