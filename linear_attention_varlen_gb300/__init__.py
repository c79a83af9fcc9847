"""Chunked Gated DeltaNet over packed varlen batches on GB300 (sm_103a).

A thin binding over the C ABI declared in include/gdn.h: argument marshalling
only. Every step of the computation runs in the CUDA library
`_build/libgdn_gb300.so`; if that library is missing, every call raises.
PyTorch is used for device memory and streams: a call runs on `stream` (the current one by default), and outputs and
workspaces that are not given are allocated for it. Inputs of another stream are the caller's to order and to keep.

    import linear_attention_varlen_gb300 as gdn
    out, final_state = gdn.chunk_fwd(q, k, v, g, beta, cu_seqlens)
    grads = gdn.chunk_bwd(q, k, v, g, beta, cu_seqlens, dout)

Beside the delta rule: decayed linear attention (la_*), the norm (rmsnorm_*), and a state-space block's short convolution
with its activation (conv_*), selective scan (ssm_*) and norm with its gate (gated_rmsnorm_*).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libgdn_gb300.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, GDN_ERR_WORKSPACE = 0, -1, -2, -3, -4, -5
MODE_EXACT, MODE_TRUNCATE = 0, 1
HEAD_DIM = 128
CHUNK = 64

# Every symbol include/gdn.h declares.
EXPORTS = ("gdn_default_options", "gdn_fwd_workspace_size", "gdn_bwd_workspace_size", "gdn_chunk_fwd",
           "gdn_chunk_bwd", "gdn_workspace_status", "gdn_status_string", "gdn_plan_host", "gdn_chunk_fwd_noalloc",
           "gdn_noalloc_scratch_bytes", "gdn_noalloc_status", "gdn_fwd_check_args", "gdn_bwd_check_args",
           "gdn_decode_step", "gdn_conv_workspace_size", "gdn_conv_fwd", "gdn_conv_bwd", "gdn_la_workspace_size",
           "gdn_la_fwd", "gdn_la_bwd", "gdn_la_decode_step", "gdn_rmsnorm_fwd", "gdn_rmsnorm_workspace_size",
           "gdn_rmsnorm_bwd", "gdn_conv_act_workspace_size", "gdn_conv_act_fwd", "gdn_conv_act_bwd",
           "gdn_conv_decode_step", "gdn_ssm_workspace_size", "gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_ssm_decode_step",
           "gdn_gated_rmsnorm_fwd", "gdn_gated_rmsnorm_workspace_size", "gdn_gated_rmsnorm_bwd", "gdn_test_withhold")


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class COptions(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("trunc_log_threshold", ctypes.c_float),
                ("segment_chunks", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_int32),
                ("stage_events", ctypes.c_void_p), ("flag_wait_us", ctypes.c_int32)]


NUM_STAGES = 11
(STAGE_PLAN, STAGE_KKT_SOLVE, STAGE_SPLIT, STAGE_CHAIN, STAGE_REV_CHAIN, STAGE_GRADS, STAGE_DINIT, STAGE_DQ,
 STAGE_OUT, STAGE_L2NORM, STAGE_L2NORM_BWD) = range(11)
FLAG_SAVE_FOR_BWD = 1  # forward of a training step: keep the records for the backward
FLAG_REUSE_FWD = 2     # backward: use the records of a FLAG_SAVE_FOR_BWD forward instead of recomputing
FLAG_TEST_WITHHOLD_FORK = 4  # forward, tests of the bounded waits only: forked documents never get their start
FLAG_L2NORM_QK = 8     # q and k come unnormalised: the library scales each row to unit L2 norm (both directions)
FLAG_FP16_INPUTS = 16  # q, k, v (and dout) are fp16; set by the calls below when the tensors are float16


@dataclass
class Options:
    """Mirror of gdn_options. mode: "exact" (default) or "truncate". save_for_backward (forward) and
    reuse_forward (backward) set the two gdn_flags of a training step that shares one workspace."""
    mode: str = "exact"
    trunc_log_threshold: float = -10.0
    segment_chunks: int = 0
    scale: float = 1.0
    stage_events: Optional[object] = None  # optional list of 2 * NUM_STAGES timing torch.cuda.Event (or None)
    save_for_backward: bool = False
    reuse_forward: bool = False
    l2norm_qk: bool = False          # q and k unnormalised: normalise each row first (forward and backward)
    fp16_inputs: bool = False        # q, k, v (and dout) in fp16 (the tensor calls below set it from the dtype)
    flag_wait_us: int = 0            # limit of a wait for another item's published state (0 = about 2 s)
    test_withhold_fork: bool = False  # tests only: make the waits of forked documents run out

    def c(self) -> COptions:
        m = {"exact": MODE_EXACT, "truncate": MODE_TRUNCATE}[self.mode]
        ev = None
        if self.stage_events is not None:
            # None entries are not recorded (each recorded event costs a few microseconds of stream time)
            handles = [0 if e is None else int(e.cuda_event) for e in self.stage_events]
            given = [e for e in self.stage_events if e is not None]
            if len(handles) != 2 * NUM_STAGES or not all(int(e.cuda_event) for e in given):
                raise ValueError("stage_events: 2 * NUM_STAGES entries, each None or a recorded timing event")
            self._ev_array = (ctypes.c_void_p * len(handles))(*handles)
            ev = ctypes.cast(self._ev_array, ctypes.c_void_p)
        flags = ((FLAG_SAVE_FOR_BWD if self.save_for_backward else 0) | (FLAG_REUSE_FWD if self.reuse_forward else 0)
                 | (FLAG_TEST_WITHHOLD_FORK if self.test_withhold_fork else 0)
                 | (FLAG_L2NORM_QK if self.l2norm_qk else 0)
                 | (FLAG_FP16_INPUTS if self.fp16_inputs else 0))
        return COptions(m, float(self.trunc_log_threshold), int(self.segment_chunks), float(self.scale), flags, ev,
                        int(self.flag_wait_us))


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return LIB_PATH


def load(path: Optional[str] = None):
    """Open the compiled library (no fallback: raises if it is missing) and declare signatures."""
    global _lib
    if _lib is not None and path is None:  # set once its signatures are declared
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"GDN CUDA library not built: {p} is missing (run linear_attention_varlen_gb300.build)")
        lib = ctypes.CDLL(p)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        OP = ctypes.POINTER(COptions)
        lib.gdn_default_options.argtypes = [OP]
        lib.gdn_default_options.restype = None
        lib.gdn_fwd_workspace_size.argtypes = [I, I, I, I, OP]
        lib.gdn_fwd_workspace_size.restype = Z
        lib.gdn_bwd_workspace_size.argtypes = [I, I, I, I, OP]
        lib.gdn_bwd_workspace_size.restype = Z
        lib.gdn_chunk_fwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, P, P, Z, OP, P]
        lib.gdn_chunk_fwd.restype = I
        lib.gdn_chunk_bwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, P, P, P, P, Z, OP, P]
        lib.gdn_chunk_bwd.restype = I
        lib.gdn_workspace_status.argtypes = [P, P]
        lib.gdn_workspace_status.restype = I
        lib.gdn_status_string.argtypes = [I]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_plan_host.argtypes = [P, I, I, I, P, I, OP, I, P, P, P, I, P, I, P]
        lib.gdn_plan_host.restype = I
        lib.gdn_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, P, OP, P]
        lib.gdn_chunk_fwd_noalloc.restype = I
        lib.gdn_noalloc_scratch_bytes.argtypes = []
        lib.gdn_noalloc_scratch_bytes.restype = Z
        lib.gdn_noalloc_status.argtypes = [I, P]
        lib.gdn_noalloc_status.restype = I
        lib.gdn_fwd_check_args.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, P, P, Z, OP]
        lib.gdn_fwd_check_args.restype = I
        lib.gdn_bwd_check_args.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, P, P, P, P, Z, OP]
        lib.gdn_bwd_check_args.restype = I
        lib.gdn_decode_step.argtypes = [P, P, P, P, P, I, I, I, I, P, P, I, P, P, OP, P]
        lib.gdn_decode_step.restype = I
        lib.gdn_conv_workspace_size.argtypes = [I, I, I, I]
        lib.gdn_conv_workspace_size.restype = Z
        lib.gdn_conv_fwd.argtypes = [P, P, P, P, I, I, I, P, P, I, P, P, P, Z, P]
        lib.gdn_conv_fwd.restype = I
        lib.gdn_conv_bwd.argtypes = [P, P, P, P, I, I, I, P, P, I, P, P, P, P, P, P, P, Z, P]
        lib.gdn_conv_bwd.restype = I
        F, L = ctypes.c_float, ctypes.c_int64
        lib.gdn_la_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.gdn_la_workspace_size.restype = Z
        lib.gdn_la_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, P, I, F, P, P, P, Z, P]
        lib.gdn_la_fwd.restype = I
        lib.gdn_la_bwd.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, P, I, F, P, P, P, P, P, P, P, Z, P]
        lib.gdn_la_bwd.restype = I
        lib.gdn_la_decode_step.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P, I, F, P, P, P]
        lib.gdn_la_decode_step.restype = I
        lib.gdn_rmsnorm_fwd.argtypes = [P, P, P, L, I, I, I, F, P, P, I, P, P]
        lib.gdn_rmsnorm_fwd.restype = I
        lib.gdn_rmsnorm_workspace_size.argtypes = [L, I, I]
        lib.gdn_rmsnorm_workspace_size.restype = Z
        lib.gdn_rmsnorm_bwd.argtypes = [P, P, P, P, L, I, I, I, F, P, P, P, Z, P]
        lib.gdn_rmsnorm_bwd.restype = I
        lib.gdn_conv_act_workspace_size.argtypes = [I, I, I, I]
        lib.gdn_conv_act_workspace_size.restype = Z
        lib.gdn_conv_act_fwd.argtypes = [P, L, P, P, P, I, I, I, I, I, P, P, I, P, P, P, Z, P]
        lib.gdn_conv_act_fwd.restype = I
        lib.gdn_conv_act_bwd.argtypes = [P, L, P, P, P, I, I, I, I, I, P, P, I, P, L, P, P, P, P, P, P, Z, P]
        lib.gdn_conv_act_bwd.restype = I
        lib.gdn_conv_decode_step.argtypes = [P, L, P, P, I, I, I, I, P, P, I, P, P, P]
        lib.gdn_conv_decode_step.restype = I
        lib.gdn_ssm_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.gdn_ssm_workspace_size.restype = Z
        lib.gdn_ssm_fwd.argtypes = [P] * 9 + [I] * 6 + [P, I, P, P, I, P, P, P, Z, P]
        lib.gdn_ssm_fwd.restype = I
        lib.gdn_ssm_bwd.argtypes = [P] * 9 + [I] * 6 + [P, I, P, P, I] + [P] * 12 + [Z, P]
        lib.gdn_ssm_bwd.restype = I
        lib.gdn_ssm_decode_step.argtypes = [P] * 8 + [I] * 5 + [P, I, P, P, I, P, P, P]
        lib.gdn_ssm_decode_step.restype = I
        lib.gdn_gated_rmsnorm_fwd.argtypes = [P, L, P, L, P, L, I, I, I, I, I, I, F, P, P]
        lib.gdn_gated_rmsnorm_fwd.restype = I
        lib.gdn_gated_rmsnorm_workspace_size.argtypes = [L, I, I, I]
        lib.gdn_gated_rmsnorm_workspace_size.restype = Z
        lib.gdn_gated_rmsnorm_bwd.argtypes = [P, L, P, L, P, P, L, L, I, I, I, I, I, I, F, P, P, P, P, Z, P]
        lib.gdn_gated_rmsnorm_bwd.restype = I
        lib.gdn_test_withhold.argtypes = [I, I]
        lib.gdn_test_withhold.restype = I
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load().gdn_status_string(int(status)).decode()
    except RuntimeError:
        return {0: "GDN_OK", -1: "GDN_ERR_INVALID_ARG", -2: "GDN_ERR_UNSUPPORTED", -3: "GDN_ERR_CUDA",
                -4: "GDN_ERR_TIMEOUT", -5: "GDN_ERR_WORKSPACE"}.get(int(status), "GDN_ERR_UNKNOWN")


def _opts(options: Optional[Options]) -> COptions:
    return (options or Options()).c()


def _half_dtype(q):
    """bf16 or fp16 inputs: the dtype of q decides, k and v (and dout) must match it."""
    torch = _torch()
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q: expected a bfloat16 or float16 tensor")
    return q.dtype


def _with_dtype(options: Optional[Options], half) -> Options:
    import dataclasses
    torch = _torch()
    base = options or Options()
    return dataclasses.replace(base, fp16_inputs=(half == torch.float16))


def fwd_workspace_size(N: int, T: int, H_k: int, H_v: int, options: Optional[Options] = None) -> int:
    o = _opts(options)
    return int(load().gdn_fwd_workspace_size(N, T, H_k, H_v, ctypes.byref(o)))


def bwd_workspace_size(N: int, T: int, H_k: int, H_v: int, options: Optional[Options] = None) -> int:
    o = _opts(options)
    return int(load().gdn_bwd_workspace_size(N, T, H_k, H_v, ctypes.byref(o)))


def plan_host(cu_seqlens, H_v: int, init_idx=None, n_init: int = 0, options: Optional[Options] = None,
              num_sms: int = 152):
    """Run the exported host planner on host arrays; returns (chunks [n,3], segments [s,4], seg_len)."""
    import numpy as np
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    N = cu.shape[0] - 1
    T = int(cu[-1])
    ii = None if init_idx is None else np.ascontiguousarray(init_idx, dtype=np.int32)
    mc = T // CHUNK + N + 1
    ms = mc + N + 1
    cs, ct, cl = (np.zeros(mc, np.int32) for _ in range(3))
    si = np.zeros(4 * ms, np.int32)
    cnt = np.zeros(3, np.int32)
    o = _opts(options)
    ptr = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    rc = load().gdn_plan_host(ptr(cu), N, T, H_v, ptr(ii), n_init, ctypes.byref(o), num_sms, ptr(cs), ptr(ct),
                              ptr(cl), mc, ptr(si), ms, ptr(cnt))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_plan_host")
    nc, ns, L = int(cnt[0]), int(cnt[1]), int(cnt[2])
    chunks = np.stack([cs[:nc], ct[:nc], cl[:nc]], axis=1)
    return chunks, si[:4 * ns].reshape(ns, 4), L


# ----------------------------------------------------------------------------- torch-facing calls


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    if stream is not None:
        return stream.cuda_stream
    c = _torch()._C  # the current stream's handle without building a Stream object (a few microseconds)
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _empty_on(stream):
    """torch.empty for a call on `stream` beside the current one. The memory comes from that stream's share of the
    allocator: the current stream's might still be in use by earlier work there, and a workspace, released when the
    call returns, could be given away while the kernels are at work. Nor is it reused before the current stream, which
    is likely to read the outputs, has gone past their release."""
    torch = _torch()

    def empty(shape, dtype, device):
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
        if t.numel():
            t.record_stream(torch.cuda.current_stream(t.device))
        return t
    return empty


def _check(t, name, dtype, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor")
    if shape is not None and t.shape != shape:  # a torch.Size is a tuple
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def chunk_fwd(q, k, v, g, beta, cu_seqlens, init_idx=None, initial_state=None, options: Optional[Options] = None,
              out=None, final_state=None, workspace=None, stream=None):
    """Forward over a packed batch. Shapes: q, k [T, Hk, 128] bf16; v [T, Hv, 128] bf16;
    g, beta [T, Hv] fp32; cu_seqlens [N+1] int32 (device); init_idx [N] int32 or None;
    initial_state [n_init, Hv, 128, 128] fp32 or None. Returns (out, final_state).
    With options.save_for_backward the workspace (allocated here when not given, of the backward's
    size) keeps the records for chunk_bwd(..., options with reuse_forward, workspace=the same)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    T, Hk, D = q.shape
    Hv = v.shape[1]
    N = cu_seqlens.shape[0] - 1
    half = _half_dtype(q)
    options = _with_dtype(options, half)
    _check(q, "q", half, (T, Hk, D))
    _check(k, "k", half, (T, Hk, D))
    _check(v, "v", half, (T, Hv, D))
    _check(g, "g", torch.float32, (T, Hv))
    _check(beta, "beta", torch.float32, (T, Hv))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    n_init = 0
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32)
        n_init = initial_state.shape[0]
    if init_idx is not None:
        _check(init_idx, "init_idx", torch.int32, (N,))
    dev = q.device
    if out is None:
        out = empty((T, Hv, D), dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = empty((N, Hv, D, D), dtype=torch.float32, device=dev)
    o = _opts(options)
    need = int(load().gdn_fwd_workspace_size(N, T, Hk, Hv, ctypes.byref(o)))
    if workspace is None:
        workspace = empty(need, dtype=torch.uint8, device=dev)
    rc = load().gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, Hk, Hv, D,
                              _ptr(init_idx), _ptr(initial_state), n_init, _ptr(out), _ptr(final_state),
                              _ptr(workspace), workspace.numel(), ctypes.byref(o), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_fwd")
    return out, final_state


def chunk_bwd(q, k, v, g, beta, cu_seqlens, dout, dfinal_state=None, init_idx=None, initial_state=None,
              options: Optional[Options] = None, workspace=None, stream=None, grads=None):
    """Backward. Returns dict of fp32 gradients dq, dk, dv, dg, dbeta and dinit (None without a pool).
    With options.reuse_forward, `workspace` must be the one a save_for_backward forward of the same
    inputs used. `grads` may hold preallocated fp32 outputs (keys dq, dk, dv, dg, dbeta, dinit)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if options is not None and options.reuse_forward and workspace is None:
        raise ValueError("reuse_forward needs the workspace of the save_for_backward forward")
    T, Hk, D = q.shape
    Hv = v.shape[1]
    N = cu_seqlens.shape[0] - 1
    half = _half_dtype(q)
    options = _with_dtype(options, half)
    _check(q, "q", half, (T, Hk, D))
    _check(k, "k", half, (T, Hk, D))
    _check(v, "v", half, (T, Hv, D))
    _check(dout, "dout", half, (T, Hv, D))
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", torch.float32, (N, Hv, D, D))
    n_init = 0 if initial_state is None else initial_state.shape[0]
    dev = q.device
    grads = grads or {}
    f32 = torch.float32

    def out_buf(key, shape):
        t = grads.get(key)
        if t is None:
            return empty(shape, dtype=f32, device=dev)
        return _check(t, key, f32, shape)
    dq = out_buf("dq", q.shape)
    dk = out_buf("dk", k.shape)
    dv = out_buf("dv", v.shape)
    dg = out_buf("dg", (T, Hv))
    db = out_buf("dbeta", (T, Hv))
    dinit = out_buf("dinit", initial_state.shape) if n_init > 0 else None
    o = _opts(options)
    need = int(load().gdn_bwd_workspace_size(N, T, Hk, Hv, ctypes.byref(o)))
    if workspace is None:
        workspace = empty(need, dtype=torch.uint8, device=dev)
    rc = load().gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, Hk, Hv, D,
                              _ptr(init_idx), _ptr(initial_state), n_init, _ptr(dout), _ptr(dfinal_state),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(db), _ptr(dinit), _ptr(workspace),
                              workspace.numel(), ctypes.byref(o), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_bwd")
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, dinit=dinit)


def decode_step(q, k, v, g, beta, state_pool, state_idx, options: Optional[Options] = None, out=None, status=None,
                stream=None):
    """One decode token per sequence, in place on the state pool. Shapes: q, k [B, Hk, 128] bf16;
    v [B, Hv, 128] bf16; g, beta [B, Hv] fp32; state_pool [n_pool, Hv, 128, 128] fp32 (updated);
    state_idx [B] int32 (distinct entries of the pool). Returns out [B, Hv, 128] bf16. `status`: an
    optional int32 device tensor of one element that receives GDN_ERR_INVALID_ARG for out-of-range
    indices (not cleared here)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    B, Hk, D = q.shape
    Hv = v.shape[1]
    half = _half_dtype(q)
    options = _with_dtype(options, half)
    _check(q, "q", half, (B, Hk, D))
    _check(k, "k", half, (B, Hk, D))
    _check(v, "v", half, (B, Hv, D))
    _check(g, "g", torch.float32, (B, Hv))
    _check(beta, "beta", torch.float32, (B, Hv))
    _check(state_idx, "state_idx", torch.int32, (B,))
    _check(state_pool, "state_pool", torch.float32)
    if state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (Hv, D, D):
        raise ValueError("state_pool: expected [n_pool, Hv, 128, 128]")
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    if out is None:
        out = empty((B, Hv, D), dtype=torch.bfloat16, device=q.device)
    o = _opts(options)
    rc = load().gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), B, Hk, Hv, D, _ptr(state_idx),
                                _ptr(state_pool), state_pool.shape[0], _ptr(out), _ptr(status), ctypes.byref(o),
                                _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_decode_step")
    return out


ACTIVATIONS = {"none": 0, "silu": 1}


def conv_workspace_size(N: int, T: int, C: int, backward: bool = False, activation=None) -> int:
    size = load().gdn_conv_workspace_size if activation is None else load().gdn_conv_act_workspace_size
    return int(size(N, T, C, 1 if backward else 0))


def _tokens(t, name, dtype, shape, align=1):
    """A tensor whose tokens (the first dimension) may be further apart than they need, the rest contiguous. Returns
    the elements between tokens, 0 when contiguous."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    strides, need = t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if strides[i] != need and shape[i] > 1:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        need *= shape[i]
    st = strides[0]
    if st < need or st % align != 0:
        raise ValueError(f"{name}: tokens must be a multiple of {align} elements apart, at least {need}")
    return st


def _conv_act_inputs(x, w, cu_seqlens, bias, init_idx, conv_init, activation, step=False):
    torch = _torch()
    if activation not in ACTIVATIONS:
        raise ValueError(f'activation: expected {"" if step else "None, "}"none" or "silu"')
    code = _dtype_code(x, "x", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32))
    T, C = x.shape
    xs = _tokens(x, "x", x.dtype, (T, C), 16 // x.element_size())
    _check(w, "w", torch.float32, (C, 4))
    if bias is not None:
        _check(bias, "bias", torch.float32, (C,))
    if step:
        return T, C, code, ACTIVATIONS[activation], xs
    N = cu_seqlens.shape[0] - 1
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    if init_idx is not None:
        _check(init_idx, "init_idx", torch.int32, (N,))
    n_init = 0
    if conv_init is not None:
        n_init = conv_init.shape[0]
        _check(conv_init, "conv_init", x.dtype, (n_init, 3, C))
    return T, C, N, n_init, code, ACTIVATIONS[activation], xs


def conv_fwd(x, w, cu_seqlens, bias=None, init_idx=None, conv_init=None, y=None, final_tail=None, workspace=None,
             stream=None, activation=None):
    """Width-4 causal convolution over packed documents. x [T, C] bf16; w [C, 4] fp32; bias [C] fp32 or
    None; cu_seqlens [N+1] int32; init_idx [N] int32 or None; conv_init [n_init, 3, C] bf16 or None.
    Returns (y [T, C] bf16, final_tail [N, 3, C] bf16).

    With activation "silu" (or "none") x may be fp16 or fp32 too and its tokens apart (a view into a
    projection), C is at most 2^23, and y, conv_init and final_tail are of x's type; the workspace is then
    conv_workspace_size(..., activation=activation) bytes."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if activation is not None:
        T, C, N, n_init, code, act, xs = _conv_act_inputs(x, w, cu_seqlens, bias, init_idx, conv_init, activation)
        y = empty((T, C), dtype=x.dtype, device=x.device) if y is None else _check(y, "y", x.dtype, (T, C))
        if final_tail is None:
            final_tail = empty((N, 3, C), dtype=x.dtype, device=x.device)
        else:
            _check(final_tail, "final_tail", x.dtype, (N, 3, C))
        if workspace is None:
            workspace = empty(conv_workspace_size(N, T, C, False, activation), dtype=torch.uint8, device=x.device)
        rc = load().gdn_conv_act_fwd(_ptr(x), xs, _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, C, code, act,
                                     _ptr(init_idx), _ptr(conv_init), n_init, _ptr(y), _ptr(final_tail),
                                     _ptr(workspace), workspace.numel(), _stream_handle(stream))
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_conv_act_fwd")
        return y, final_tail
    T, C = x.shape
    N = cu_seqlens.shape[0] - 1
    _check(x, "x", torch.bfloat16, (T, C))
    _check(w, "w", torch.float32, (C, 4))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    if bias is not None:
        _check(bias, "bias", torch.float32, (C,))
    if init_idx is not None:
        _check(init_idx, "init_idx", torch.int32, (N,))
    n_init = 0
    if conv_init is not None:
        _check(conv_init, "conv_init", torch.bfloat16)
        n_init = conv_init.shape[0]
    if y is None:
        y = empty((T, C), dtype=torch.bfloat16, device=x.device)
    if final_tail is None:
        final_tail = empty((N, 3, C), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = empty(conv_workspace_size(N, T, C), dtype=torch.uint8, device=x.device)
    rc = load().gdn_conv_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, C, _ptr(init_idx), _ptr(conv_init),
                             n_init, _ptr(y), _ptr(final_tail), _ptr(workspace), workspace.numel(),
                             _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_conv_fwd")
    return y, final_tail


def conv_bwd(x, w, cu_seqlens, dy, bias=None, init_idx=None, conv_init=None, dfinal_tail=None, workspace=None,
             stream=None, activation=None):
    """Backward of conv_fwd. Returns dict dx [T, C], dw [C, 4], dbias [C] (None without bias),
    dconv_init [n_init, 3, C] (None without a pool), all fp32. `activation` as given to conv_fwd; with it dy may be
    strided as x."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    T, C = x.shape
    N = cu_seqlens.shape[0] - 1
    if activation is not None:
        T, C, N, n_init, code, act, xs = _conv_act_inputs(x, w, cu_seqlens, bias, init_idx, conv_init, activation)
        gs = _tokens(dy, "dy", x.dtype, (T, C), 16 // x.element_size())
        if dfinal_tail is not None:
            _check(dfinal_tail, "dfinal_tail", torch.float32, (N, 3, C))
        f32 = dict(dtype=torch.float32, device=x.device)
        dx, dw = empty((T, C), **f32), empty((C, 4), **f32)
        dbias = empty((C,), **f32) if bias is not None else None
        dci = empty((n_init, 3, C), **f32) if n_init > 0 else None
        if workspace is None:
            workspace = empty(conv_workspace_size(N, T, C, True, activation), dtype=torch.uint8, device=x.device)
        rc = load().gdn_conv_act_bwd(_ptr(x), xs, _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, C, code, act,
                                     _ptr(init_idx), _ptr(conv_init), n_init, _ptr(dy), gs, _ptr(dfinal_tail), _ptr(dx),
                                     _ptr(dw), _ptr(dbias), _ptr(dci), _ptr(workspace), workspace.numel(),
                                     _stream_handle(stream))
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_conv_act_bwd")
        return dict(dx=dx, dw=dw, dbias=dbias, dconv_init=dci)
    _check(dy, "dy", torch.bfloat16, (T, C))
    if dfinal_tail is not None:
        _check(dfinal_tail, "dfinal_tail", torch.float32, (N, 3, C))
    n_init = 0 if conv_init is None else conv_init.shape[0]
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = empty((T, C), **f32)
    dw = empty((C, 4), **f32)
    dbias = empty((C,), **f32) if bias is not None else None
    dci = empty((n_init, 3, C), **f32) if n_init > 0 else None
    if workspace is None:
        workspace = empty(conv_workspace_size(N, T, C, True), dtype=torch.uint8, device=x.device)
    rc = load().gdn_conv_bwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(cu_seqlens), N, T, C, _ptr(init_idx), _ptr(conv_init),
                             n_init, _ptr(dy), _ptr(dfinal_tail), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(dci),
                             _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_conv_bwd")
    return dict(dx=dx, dw=dw, dbias=dbias, dconv_init=dci)


def conv_decode_step(x, w, tail_pool, state_idx, bias=None, activation="none", y=None, status=None, stream=None):
    """One token per sequence of the convolution with its activation ("none" or "silu"), in place on a pool of tails.
    x [B, C] (bf16, fp16 or fp32; sequences may be strided); w [C, 4], bias [C] fp32; tail_pool [n_pool, 3, C] of x's
    type (updated); state_idx [B] int32 (distinct entries); status as in decode_step. Returns y [B, C]."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    B, C, code, act, xs = _conv_act_inputs(x, w, None, bias, None, None, activation, step=True)
    _check(state_idx, "state_idx", torch.int32, (B,))
    if tail_pool is None:
        raise ValueError("tail_pool is required")
    _check(tail_pool, "tail_pool", x.dtype, (tail_pool.shape[0], 3, C))
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    y = empty((B, C), dtype=x.dtype, device=x.device) if y is None else _check(y, "y", x.dtype, (B, C))
    rc = load().gdn_conv_decode_step(_ptr(x), xs, _ptr(w), _ptr(bias), B, C, code, act, _ptr(state_idx),
                                     _ptr(tail_pool), tail_pool.shape[0], _ptr(y), _ptr(status), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_conv_decode_step")
    return y


# ----------------------------------------------------------------------------- decayed linear attention

DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
QUANT = {"none": 0, None: 0, "row": 1, "group": 2}
NORM_GROUP = 128  # columns to one scale of quant="group"


_codes = {}


def _dtype_code(t, name, allowed):
    if not _codes:
        torch = _torch()
        _codes.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32})
    code = _codes.get(t.dtype)
    if code not in allowed:
        raise ValueError(f"{name}: unsupported type {t.dtype}")
    return code


def _rows(t, name, dtype, shape):
    """A tensor [tokens, heads, 128] whose tokens may be further apart than its heads need (a view into a
    fused projection). Returns the elements between tokens, 0 when contiguous."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    n, heads, d = shape
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != d) or st[0] < heads * d or st[0] % 8 != 0:
        raise ValueError(f"{name}: the heads of a token must be contiguous and tokens a multiple of 8 elements apart")
    return st[0]


def _strides(values):
    return (ctypes.c_int64 * len(values))(*values) if any(values) else None


def la_workspace_size(N: int, T: int, H_k: int, H_v: int, has_init: bool = False, backward: bool = False) -> int:
    return int(load().gdn_la_workspace_size(N, T, H_k, H_v, 1 if has_init else 0, 1 if backward else 0))


def _la_inputs(q, k, v, log_decay, cu_seqlens, init_idx, initial_state, dout=None):
    torch = _torch()
    T, Hk, D = q.shape
    Hv = v.shape[1]
    N = cu_seqlens.shape[0] - 1
    strides = [_rows(q, "q", torch.bfloat16, (T, Hk, D)), _rows(k, "k", torch.bfloat16, (T, Hk, D)),
               _rows(v, "v", torch.bfloat16, (T, Hv, D))]
    if dout is not None:
        strides.append(_rows(dout, "dout", torch.bfloat16, (T, Hv, D)))
    _check(log_decay, "log_decay", torch.float32, (Hv,))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    n_init = 0
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32)
        if initial_state.dim() != 4 or tuple(initial_state.shape[1:]) != (Hv, D, D):
            raise ValueError("initial_state: expected [n_init, Hv, 128, 128]")
        n_init = initial_state.shape[0]
    if init_idx is not None:
        _check(init_idx, "init_idx", torch.int32, (N,))
    return T, Hk, Hv, D, N, n_init, _strides(strides)


def la_chunk_fwd(q, k, v, log_decay, cu_seqlens, init_idx=None, initial_state=None, scale: float = 1.0, out=None,
                 final_state=None, workspace=None, stream=None):
    """Decayed linear attention over a packed batch: S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale
    S_t^T q_t. Shapes: q, k [T, Hk, 128] bf16; v [T, Hv, 128] bf16 (tokens may be strided); log_decay [Hv]
    fp32; cu_seqlens, init_idx and initial_state as in chunk_fwd. Returns (out [T, Hv, 128] bf16,
    final_state [N, Hv, 128, 128] fp32)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    T, Hk, Hv, D, N, n_init, strides = _la_inputs(q, k, v, log_decay, cu_seqlens, init_idx, initial_state)
    dev = q.device
    if out is None:
        out = empty((T, Hv, D), dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", torch.bfloat16, (T, Hv, D))
    if final_state is None:
        final_state = empty((N, Hv, D, D), dtype=torch.float32, device=dev)
    else:
        _check(final_state, "final_state", torch.float32, (N, Hv, D, D))
    if workspace is None:
        workspace = empty(la_workspace_size(N, T, Hk, Hv, init_idx is not None), dtype=torch.uint8, device=dev)
    rc = load().gdn_la_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu_seqlens), N, T, Hk, Hv, D, strides,
                           _ptr(init_idx), _ptr(initial_state), n_init, float(scale), _ptr(out), _ptr(final_state),
                           _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_la_fwd")
    return out, final_state


def la_chunk_bwd(q, k, v, log_decay, cu_seqlens, dout, dfinal_state=None, init_idx=None, initial_state=None,
                 scale: float = 1.0, workspace=None, stream=None, grads=None):
    """Backward of la_chunk_fwd. Returns dict of dq, dk, dv (bf16) and dinit (fp32; None without a pool).
    `grads` may hold preallocated outputs under those keys."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if dout is None:
        raise ValueError("dout is required")
    T, Hk, Hv, D, N, n_init, strides = _la_inputs(q, k, v, log_decay, cu_seqlens, init_idx, initial_state, dout)
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", torch.float32, (N, Hv, D, D))
    dev = q.device
    grads = grads or {}

    def out_buf(key, shape, dtype):
        t = grads.get(key)
        return empty(shape, dtype=dtype, device=dev) if t is None else _check(t, key, dtype, shape)
    dq = out_buf("dq", (T, Hk, D), torch.bfloat16)
    dk = out_buf("dk", (T, Hk, D), torch.bfloat16)
    dv = out_buf("dv", (T, Hv, D), torch.bfloat16)
    dinit = out_buf("dinit", (n_init, Hv, D, D), torch.float32) if n_init > 0 else None
    if workspace is None:
        workspace = empty(la_workspace_size(N, T, Hk, Hv, init_idx is not None, True), dtype=torch.uint8, device=dev)
    rc = load().gdn_la_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu_seqlens), N, T, Hk, Hv, D, strides,
                           _ptr(init_idx), _ptr(initial_state), n_init, float(scale), _ptr(dout), _ptr(dfinal_state),
                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dinit), _ptr(workspace), workspace.numel(),
                           _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_la_bwd")
    return dict(dq=dq, dk=dk, dv=dv, dinit=dinit)


def la_decode_step(q, k, v, log_decay, state_pool, state_idx, scale: float = 1.0, out=None, status=None, stream=None):
    """One token per sequence of the decayed linear attention, in place on the state pool. q, k [B, Hk, 128],
    v [B, Hv, 128] bf16 or fp16 (sequences may be strided); log_decay [Hv] fp32; state_pool, state_idx and
    status as in decode_step. Returns out [B, Hv, 128] of the inputs' type."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    B, Hk, D = q.shape
    Hv = v.shape[1]
    code = _dtype_code(q, "q", (DTYPE_BF16, DTYPE_FP16))
    strides = _strides([_rows(q, "q", q.dtype, (B, Hk, D)), _rows(k, "k", q.dtype, (B, Hk, D)),
                        _rows(v, "v", q.dtype, (B, Hv, D))])
    _check(log_decay, "log_decay", torch.float32, (Hv,))
    _check(state_idx, "state_idx", torch.int32, (B,))
    _check(state_pool, "state_pool", torch.float32)
    if state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (Hv, D, D):
        raise ValueError("state_pool: expected [n_pool, Hv, 128, 128]")
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    if out is None:
        out = empty((B, Hv, D), dtype=q.dtype, device=q.device)
    else:
        _check(out, "out", q.dtype, (B, Hv, D))
    rc = load().gdn_la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), B, Hk, Hv, D, code, strides,
                                   _ptr(state_idx), _ptr(state_pool), state_pool.shape[0], float(scale), _ptr(out),
                                   _ptr(status), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_la_decode_step")
    return out


# ----------------------------------------------------------------------------- root-mean-square norm


def rmsnorm_fwd(x, w, residual=None, eps: float = 1e-6, quant=None, y=None, residual_out=None, scales=None,
                stream=None):
    """y = w h / sqrt(mean(h^2) + eps) with h = x + residual, per row of x [T, D] (bf16, fp16 or fp32; w [D] of
    any of them). quant: None, "row" or "group" (y in float8_e4m3fn with fp32 scales [T, 1] or
    [T, ceil(D / 128)]). Returns (y, h, scales); h is None without a residual, scales without quant.
    residual_out may be `residual` itself (in place)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if quant not in QUANT:
        raise ValueError('quant: expected None, "none", "row" or "group"')
    code, q = _dtype_code(x, "x", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32)), QUANT[quant]
    T, D = x.shape
    _check(x, "x", x.dtype, (T, D))
    wcode = _dtype_code(w, "w", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32))
    _check(w, "w", w.dtype, (D,))
    if residual is not None:
        _check(residual, "residual", x.dtype, (T, D))
        if residual_out is None:
            residual_out = empty((T, D), dtype=x.dtype, device=x.device)
        else:
            _check(residual_out, "residual_out", x.dtype, (T, D))
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    ydt = torch.float8_e4m3fn if q else x.dtype
    if y is None:
        y = empty((T, D), dtype=ydt, device=x.device)
    else:
        _check(y, "y", ydt, (T, D))
    if q:
        shape = (T, 1 if q == 1 else -(-D // NORM_GROUP))
        if scales is None:
            scales = empty(shape, dtype=torch.float32, device=x.device)
        else:
            _check(scales, "scales", torch.float32, shape)
    elif scales is not None:
        raise ValueError("scales without quant")
    rc = load().gdn_rmsnorm_fwd(_ptr(x), _ptr(residual), _ptr(w), T, D, code, wcode, float(eps), _ptr(residual_out),
                                _ptr(y), q, _ptr(scales), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_rmsnorm_fwd")
    return y, residual_out, scales


def rmsnorm_bwd(h, w, dy, dh=None, eps: float = 1e-6, dx=None, dw=None, workspace=None, stream=None):
    """Backward of rmsnorm_fwd from the h it left (x without a residual), dy the gradient of y and dh that of h
    from elsewhere. Returns (dx [T, D] of h's type: the gradient of x and of the residual, dw [D] fp32)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    code = _dtype_code(h, "h", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32))
    T, D = h.shape
    _check(h, "h", h.dtype, (T, D))
    _check(dy, "dy", h.dtype, (T, D))
    wcode = _dtype_code(w, "w", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32))
    _check(w, "w", w.dtype, (D,))
    if dh is not None:
        _check(dh, "dh", h.dtype, (T, D))
    if dx is None:
        dx = empty((T, D), dtype=h.dtype, device=h.device)
    else:
        _check(dx, "dx", h.dtype, (T, D))
    if dw is None:
        dw = empty((D,), dtype=torch.float32, device=h.device)
    else:
        _check(dw, "dw", torch.float32, (D,))
    if workspace is None:
        workspace = empty(int(load().gdn_rmsnorm_workspace_size(T, D, code)), dtype=torch.uint8, device=h.device)
    rc = load().gdn_rmsnorm_bwd(_ptr(h), _ptr(w), _ptr(dy), _ptr(dh), T, D, code, wcode, float(eps), _ptr(dx), _ptr(dw),
                                _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_rmsnorm_bwd")
    return dx, dw


# ----------------------------------------------------------------------------- selective scan


def ssm_workspace_size(N: int, T: int, C: int, S: int, G: int = 1, backward: bool = False) -> int:
    return int(load().gdn_ssm_workspace_size(N, T, C, S, G, 1 if backward else 0))


def _ssm_inputs(x, dt, a, b, c, skip, z, dt_bias, dout=None):
    torch = _torch()
    code = _dtype_code(x, "x", (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32))
    T, C = x.shape
    _, G, S = b.shape
    h = x.dtype
    strides = [_tokens(x, "x", h, (T, C)), _tokens(dt, "dt", h, (T, C)),
               0 if z is None else _tokens(z, "z", h, (T, C)),
               _tokens(b, "b", h, (T, G, S)), _tokens(c, "c", h, (T, G, S))]
    if dout is not None:
        strides.append(_tokens(dout, "dout", h, (T, C)))
    _check(a, "a", torch.float32, (C, S))
    if skip is not None:
        _check(skip, "skip", torch.float32, (C,))
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", torch.float32, (C,))
    return code, T, C, S, G, _strides(strides)


def _ssm_packed(cu_seqlens, init_idx, initial_state, C, S):
    torch = _torch()
    N = cu_seqlens.shape[0] - 1
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    n_init = 0
    if initial_state is not None:
        n_init = initial_state.shape[0]
        _check(initial_state, "initial_state", torch.float32, (n_init, C, S))
    if init_idx is not None:
        _check(init_idx, "init_idx", torch.int32, (N,))
    return N, n_init


def ssm_scan_fwd(x, dt, a, b, c, cu_seqlens, skip=None, z=None, dt_bias=None, init_idx=None, initial_state=None,
                 dt_softplus: bool = True, out=None, final_state=None, workspace=None, stream=None):
    """Selective scan over a packed batch: with step = softplus(dt + dt_bias), h = exp(step a) h + step b x,
    out = (c . h + skip x) silu(z), per channel. Shapes: x, dt, z [T, C], b, c [T, G, S] (bf16, fp16 or fp32, all the
    same; tokens may be strided; S <= 64, channel c uses maps c // (C / G)); a [C, S], skip, dt_bias [C] fp32;
    initial_state [n_init, C, S] fp32; cu_seqlens and init_idx as in chunk_fwd. Returns (out [T, C], final_state
    [N, C, S] fp32)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    code, T, C, S, G, strides = _ssm_inputs(x, dt, a, b, c, skip, z, dt_bias)
    N, n_init = _ssm_packed(cu_seqlens, init_idx, initial_state, C, S)
    dev = x.device
    out = empty((T, C), dtype=x.dtype, device=dev) if out is None else _check(out, "out", x.dtype, (T, C))
    if final_state is None:
        final_state = empty((N, C, S), dtype=torch.float32, device=dev)
    else:
        _check(final_state, "final_state", torch.float32, (N, C, S))
    if workspace is None:
        workspace = empty(ssm_workspace_size(N, T, C, S, G), dtype=torch.uint8, device=dev)
    rc = load().gdn_ssm_fwd(_ptr(x), _ptr(dt), _ptr(z), _ptr(a), _ptr(b), _ptr(c), _ptr(skip), _ptr(dt_bias),
                            _ptr(cu_seqlens), N, T, C, S, G, code, strides, 1 if dt_softplus else 0, _ptr(init_idx),
                            _ptr(initial_state), n_init, _ptr(out), _ptr(final_state), _ptr(workspace),
                            workspace.numel(), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_ssm_fwd")
    return out, final_state


def ssm_scan_bwd(x, dt, a, b, c, cu_seqlens, dout, dfinal_state=None, skip=None, z=None, dt_bias=None, init_idx=None,
                 initial_state=None, dt_softplus: bool = True, workspace=None, stream=None, grads=None):
    """Backward of ssm_scan_fwd. Returns dict of dx, ddt, dz (None without z), db, dc of x's type and da, dskip,
    ddt_bias and dinit in fp32 (None without skip, dt_bias or a pool). `grads` may hold preallocated outputs under
    those keys."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if dout is None:
        raise ValueError("dout is required")
    code, T, C, S, G, strides = _ssm_inputs(x, dt, a, b, c, skip, z, dt_bias, dout)
    N, n_init = _ssm_packed(cu_seqlens, init_idx, initial_state, C, S)
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", torch.float32, (N, C, S))
    dev, h, f32 = x.device, x.dtype, torch.float32
    grads = grads or {}

    def out_buf(key, shape, dtype, wanted=True):
        if not wanted:
            return None
        t = grads.get(key)
        return empty(shape, dtype=dtype, device=dev) if t is None else _check(t, key, dtype, shape)
    g = dict(dx=out_buf("dx", (T, C), h), ddt=out_buf("ddt", (T, C), h), dz=out_buf("dz", (T, C), h, z is not None),
             da=out_buf("da", (C, S), f32), db=out_buf("db", (T, G, S), h), dc=out_buf("dc", (T, G, S), h),
             dskip=out_buf("dskip", (C,), f32, skip is not None),
             ddt_bias=out_buf("ddt_bias", (C,), f32, dt_bias is not None),
             dinit=out_buf("dinit", (n_init, C, S), f32, n_init > 0))
    if workspace is None:
        workspace = empty(ssm_workspace_size(N, T, C, S, G, True), dtype=torch.uint8, device=dev)
    rc = load().gdn_ssm_bwd(_ptr(x), _ptr(dt), _ptr(z), _ptr(a), _ptr(b), _ptr(c), _ptr(skip), _ptr(dt_bias),
                            _ptr(cu_seqlens), N, T, C, S, G, code, strides, 1 if dt_softplus else 0, _ptr(init_idx),
                            _ptr(initial_state), n_init, _ptr(dout), _ptr(dfinal_state), _ptr(g["dx"]), _ptr(g["ddt"]),
                            _ptr(g["dz"]), _ptr(g["da"]), _ptr(g["db"]), _ptr(g["dc"]), _ptr(g["dskip"]),
                            _ptr(g["ddt_bias"]), _ptr(g["dinit"]), _ptr(workspace), workspace.numel(),
                            _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_ssm_bwd")
    return g


def ssm_decode_step(x, dt, a, b, c, state_pool, state_idx, skip=None, z=None, dt_bias=None, dt_softplus: bool = True,
                    out=None, status=None, stream=None):
    """One token per sequence of the selective scan, in place on a pool of states. x, dt, z [B, C], b, c [B, G, S]
    (sequences may be strided); state_pool [n_pool, C, S] fp32 (updated); state_idx [B] int32 (distinct entries);
    status as in decode_step. Returns out [B, C] of x's type."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    code, B, C, S, G, strides = _ssm_inputs(x, dt, a, b, c, skip, z, dt_bias)
    _check(state_idx, "state_idx", torch.int32, (B,))
    if state_pool is None:
        raise ValueError("state_pool is required")
    _check(state_pool, "state_pool", torch.float32, (state_pool.shape[0], C, S))
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    out = empty((B, C), dtype=x.dtype, device=x.device) if out is None else _check(out, "out", x.dtype, (B, C))
    rc = load().gdn_ssm_decode_step(_ptr(x), _ptr(dt), _ptr(z), _ptr(a), _ptr(b), _ptr(c), _ptr(skip), _ptr(dt_bias), B,
                                    C, S, G, code, strides, 1 if dt_softplus else 0, _ptr(state_idx), _ptr(state_pool),
                                    state_pool.shape[0], _ptr(out), _ptr(status), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_ssm_decode_step")
    return out


# ----------------------------------------------------------------------------- norm with its gate

GATE_ORDER = {"norm": 0, "gate": 1}  # what comes first


def _gnorm_inputs(x, z, w, group, first, dy=None):
    if first not in GATE_ORDER:
        raise ValueError('first: expected "norm" or "gate"')
    allowed = (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32)
    code = _dtype_code(x, "x", allowed)
    T, D = x.shape
    group = D if group is None else int(group)
    if group < 1 or D % group:
        raise ValueError(f"group: {D} columns are no multiple of {group}")
    strides = [_tokens(x, "x", x.dtype, (T, D)), _tokens(z, "z", x.dtype, (T, D))]
    if dy is not None:
        strides.append(_tokens(dy, "dy", x.dtype, (T, D)))
    wcode = _dtype_code(w, "w", allowed)
    if tuple(w.shape) not in ((group,), (D,)):
        raise ValueError(f"w: expected {group} or {D} weights, got {tuple(w.shape)}")
    _check(w, "w", w.dtype)
    return T, D, group, 1 if w.shape[0] == group else 0, GATE_ORDER[first], code, wcode, strides


def gated_rmsnorm_fwd(x, z, w, group=None, eps: float = 1e-6, first: str = "norm", y=None, stream=None):
    """The norm of each `group` consecutive columns (a head; None = the whole row) with its gate: first="norm" gives
    y = w norm(x) silu(z), first="gate" y = w norm(x silu(z)), norm(u) = u / sqrt(mean(u^2) + eps). x, z [T, D] (bf16,
    fp16 or fp32; rows may be strided); w [group] (the same for every group) or [D], of any of the types; group <=
    16384. Returns y [T, D] of x's type; it may be x or z itself, when contiguous."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    T, D, group, shared, order, code, wcode, (xs, zs) = _gnorm_inputs(x, z, w, group, first)
    y = empty((T, D), dtype=x.dtype, device=x.device) if y is None else _check(y, "y", x.dtype, (T, D))
    rc = load().gdn_gated_rmsnorm_fwd(_ptr(x), xs, _ptr(z), zs, _ptr(w), T, D, group, shared, order, code, wcode,
                                      float(eps), _ptr(y), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_gated_rmsnorm_fwd")
    return y


def gated_rmsnorm_bwd(x, z, w, dy, group=None, eps: float = 1e-6, first: str = "norm", dx=None, dz=None, dw=None,
                      workspace=None, stream=None):
    """Backward of gated_rmsnorm_fwd. Returns (dx, dz [T, D] of x's type, dw fp32 of w's shape)."""
    torch = _torch()
    empty = torch.empty if stream is None else _empty_on(stream)
    if dy is None:
        raise ValueError("dy is required")
    T, D, group, shared, order, code, wcode, (xs, zs, gs) = _gnorm_inputs(x, z, w, group, first, dy)
    dx = empty((T, D), dtype=x.dtype, device=x.device) if dx is None else _check(dx, "dx", x.dtype, (T, D))
    dz = empty((T, D), dtype=x.dtype, device=x.device) if dz is None else _check(dz, "dz", x.dtype, (T, D))
    if dw is None:
        dw = empty(tuple(w.shape), dtype=torch.float32, device=x.device)
    else:
        _check(dw, "dw", torch.float32, tuple(w.shape))
    if workspace is None:
        workspace = empty(int(load().gdn_gated_rmsnorm_workspace_size(T, D, group, code)), dtype=torch.uint8,
                          device=x.device)
    rc = load().gdn_gated_rmsnorm_bwd(_ptr(x), xs, _ptr(z), zs, _ptr(w), _ptr(dy), gs, T, D, group, shared, order, code,
                                      wcode, float(eps), _ptr(dx), _ptr(dz), _ptr(dw), _ptr(workspace),
                                      workspace.numel(), _stream_handle(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_gated_rmsnorm_bwd")
    return dx, dz, dw


@contextlib.contextmanager
def withheld_copy(copy: int, wait_us: int = 20000):
    """For testing the bounded waits only: the calls within (of this thread) leave out one of their bulk copies, so
    that the wait for it runs out after wait_us and the workspace's status word says GDN_ERR_TIMEOUT."""
    rc = load().gdn_test_withhold(copy, wait_us)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_test_withhold")
    try:
        yield
    finally:
        load().gdn_test_withhold(0, 0)


def workspace_status(workspace, stream=None) -> int:
    """Device status word of the last call that used `workspace` (synchronises the stream)."""
    return int(load().gdn_workspace_status(_ptr(workspace), _stream_handle(stream)))
