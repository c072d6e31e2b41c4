"""Thin ctypes binding of the C ABI in include/gdn.h (argument marshalling only).

Every function here takes torch tensors that already live on the GPU, checks nothing
beyond what marshalling needs, passes raw device pointers plus the current CUDA stream to
``libgdn.so`` and raises ``GdnError`` on a non-OK status. All validation and all compute
happen in the library's CUDA kernels; there is no fallback of any kind. If ``libgdn.so``
has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgdn.so")

GDN_DTYPE_F32, GDN_DTYPE_BF16 = 0, 1
STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED_SHAPE",
          3: "GDN_ERR_UNSUPPORTED_DTYPE", 4: "GDN_ERR_MISALIGNED", 5: "GDN_ERR_WORKSPACE",
          6: "GDN_ERR_CUDA", 7: "GDN_ERR_TIMEOUT", 8: "GDN_ERR_DEVICE",
          9: "GDN_ERR_NO_PAGE"}
EXPORTED = ("gdn_workspace_bytes", "gdn_segmented_pieces", "gdn_segmented_plan", "gdn_chunk_fwd",
            "gdn_segment_summary", "gdn_summary_scan", "gdn_segment_fwd", "gdn_segmented_fwd",
            "gdn_segmented_fwd_timed", "gdn_segmented_fwd_noalloc",
            "gdn_varlen_workspace_bytes", "gdn_varlen_fwd", "gdn_varlen_fwd_timed",
            "gdn_state_grad_summary", "gdn_state_grad_scan", "gdn_chunk_bwd_workspace_bytes",
            "gdn_chunk_bwd", "gdn_chunk_bwd_timed",
            "gdn_recurrent_workspace_bytes", "gdn_recurrent_fwd",
            "gdn_cache_workspace_bytes", "gdn_cache_copy", "gdn_cache_fork", "gdn_cache_free",
            "gdn_cache_compact", "gdn_norm_fwd", "gdn_norm_bwd_workspace_bytes", "gdn_norm_bwd",
            "gdn_linear_workspace_bytes", "gdn_linear_fwd", "gdn_linear_bwd", "gdn_linear_recurrent_fwd",
            "gdn_qk_norm_fwd", "gdn_qk_norm_bwd_workspace_bytes", "gdn_qk_norm_bwd",
            "gdn_status_string", "gdn_check_device_error", "gdn_selftest_wait_timeout")


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({lib().gdn_status_string(status).decode()})")


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("K", ctypes.c_int), ("V", ctypes.c_int), ("chunk", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("decay_first", ctypes.c_int), ("gate_k", ctypes.c_int)]


class QkProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("K", ctypes.c_int), ("R", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong)]


_lib = None
_P = ctypes.c_void_p


def lib():
    """Load libgdn.so (raises OSError if it is missing: build it with __graft_entry__.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"libgdn.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        pp = ctypes.POINTER(Problem)
        L.gdn_workspace_bytes.argtypes = [pp, ctypes.c_int]
        L.gdn_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_segmented_pieces.argtypes = [pp, ctypes.c_int]
        L.gdn_segmented_pieces.restype = ctypes.c_int
        L.gdn_segmented_plan.argtypes = [pp, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_int)]
        L.gdn_segmented_plan.restype = ctypes.c_int
        L.gdn_segment_fwd.argtypes = [pp, ctypes.c_int] + [_P] * 9 + [ctypes.c_size_t, _P]
        L.gdn_chunk_fwd.argtypes = [pp] + [_P] * 9 + [ctypes.c_size_t, _P]
        L.gdn_segment_summary.argtypes = [pp, ctypes.c_int] + [_P] * 7 + [ctypes.c_size_t, _P]
        L.gdn_summary_scan.argtypes = [pp, ctypes.c_int] + [_P] * 5
        L.gdn_segmented_fwd.argtypes = [pp, ctypes.c_int] + [_P] * 10 + [ctypes.c_size_t, _P]
        L.gdn_segmented_fwd_timed.argtypes = ([pp, ctypes.c_int] + [_P] * 10 +
                                              [ctypes.c_size_t, _P, _P])
        L.gdn_segmented_fwd_noalloc.argtypes = [pp, ctypes.c_int] + [_P] * 10
        L.gdn_varlen_workspace_bytes.argtypes = [pp, ctypes.c_int]
        L.gdn_varlen_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_varlen_fwd.argtypes = [pp, ctypes.c_int] + [_P] * 10 + [ctypes.c_size_t, _P]
        L.gdn_varlen_fwd_timed.argtypes = ([pp, ctypes.c_int] + [_P] * 10 +
                                           [ctypes.c_size_t, _P, _P])
        L.gdn_state_grad_summary.argtypes = [pp, ctypes.c_int] + [_P] * 8
        L.gdn_state_grad_scan.argtypes = [pp, ctypes.c_int] + [_P] * 5
        L.gdn_chunk_bwd_workspace_bytes.argtypes = [pp, ctypes.c_int]
        L.gdn_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_chunk_bwd.argtypes = [pp, ctypes.c_int] + [_P] * 15 + [ctypes.c_size_t, _P]
        L.gdn_chunk_bwd_timed.argtypes = L.gdn_chunk_bwd.argtypes + [_P]
        L.gdn_recurrent_workspace_bytes.argtypes = [ctypes.c_int]
        L.gdn_recurrent_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_recurrent_fwd.argtypes = ([pp, ctypes.c_int, ctypes.c_int] + [_P] * 7 + [ctypes.c_int] +
                                        [_P] * 2 + [ctypes.c_int] + [_P] * 2 + [ctypes.c_size_t, _P])
        L.gdn_cache_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
        L.gdn_cache_workspace_bytes.restype = ctypes.c_size_t
        pages = [_P, ctypes.c_int, ctypes.c_int, ctypes.c_size_t]
        ws = [_P, ctypes.c_size_t, _P]
        L.gdn_cache_copy.argtypes = pages + [ctypes.c_int, _P, _P] + ws
        L.gdn_cache_fork.argtypes = pages + [_P, ctypes.c_int, _P, _P, ctypes.c_int] + ws
        L.gdn_cache_free.argtypes = [ctypes.c_int, _P, ctypes.c_int, _P] + ws
        L.gdn_cache_compact.argtypes = pages + [_P, ctypes.c_int, _P, _P, _P] + ws
        rows = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float]
        L.gdn_norm_fwd.argtypes = rows + [_P] * 6
        L.gdn_norm_bwd_workspace_bytes.argtypes = [ctypes.c_longlong, ctypes.c_int]
        L.gdn_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_norm_bwd.argtypes = rows + [_P] * 9 + ws
        L.gdn_linear_workspace_bytes.argtypes = [pp, ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.gdn_linear_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_linear_fwd.argtypes = [pp, ctypes.c_int, ctypes.c_int] + [_P] * 8 + ws
        L.gdn_linear_bwd.argtypes = [pp, ctypes.c_int, ctypes.c_int] + [_P] * 12 + ws
        L.gdn_linear_recurrent_fwd.argtypes = ([pp, ctypes.c_int, ctypes.c_int] + [_P] * 6 + [ctypes.c_int] +
                                               [_P] * 2 + [ctypes.c_int, _P] + ws)
        qk = ctypes.POINTER(QkProblem)
        L.gdn_qk_norm_fwd.argtypes = [qk] + [_P] * 9
        L.gdn_qk_norm_bwd_workspace_bytes.argtypes = [ctypes.c_int]
        L.gdn_qk_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_qk_norm_bwd.argtypes = [qk] + [_P] * 12 + ws
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_check_device_error.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint)]
        L.gdn_selftest_wait_timeout.argtypes = [_P, ctypes.c_longlong, _P]
        for fn in ("gdn_chunk_fwd", "gdn_segment_summary", "gdn_summary_scan", "gdn_segment_fwd",
                   "gdn_segmented_fwd", "gdn_segmented_fwd_timed", "gdn_segmented_fwd_noalloc",
                   "gdn_varlen_fwd", "gdn_varlen_fwd_timed", "gdn_check_device_error",
                   "gdn_selftest_wait_timeout", "gdn_state_grad_summary", "gdn_state_grad_scan",
                   "gdn_chunk_bwd", "gdn_chunk_bwd_timed", "gdn_recurrent_fwd", "gdn_cache_copy",
                   "gdn_cache_fork", "gdn_cache_free", "gdn_cache_compact", "gdn_norm_fwd",
                   "gdn_norm_bwd", "gdn_linear_fwd", "gdn_linear_bwd", "gdn_linear_recurrent_fwd",
                   "gdn_qk_norm_fwd", "gdn_qk_norm_bwd"):
            getattr(L, fn).restype = ctypes.c_int
        _lib = L
    return _lib


class _Codes(dict):
    def __missing__(self, dtype):
        import torch
        self.update({torch.float32: GDN_DTYPE_F32, torch.bfloat16: GDN_DTYPE_BF16})
        return dict.get(self, dtype, 99)   # the library rejects it with GDN_ERR_UNSUPPORTED_DTYPE


_CODES = _Codes()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return GDN_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return GDN_DTYPE_BF16
    return 99   # the library rejects it with GDN_ERR_UNSUPPORTED_DTYPE


def problem(q_or_k, v, o=None, chunk: int = 64, decay_first: bool = False, g=None) -> Problem:
    """The problem description of these tensors; g (optional) sets gate_k when it carries
    one gate per key channel ([B, T, H, K])."""
    B, T, H, K = q_or_k.shape
    V = v.shape[-1]
    out = GDN_DTYPE_F32 if o is None else _dtype_code(o)
    gate_k = int(g is not None and g.dim() == 4)
    return Problem(B, T, H, K, V, chunk, _dtype_code(q_or_k), out, int(decay_first), gate_k)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        # the current stream's handle; without a stream object around it where this torch has a way to that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status: int, where: str):
    if status != 0:
        raise GdnError(status, where)


def workspace_bytes(prob: Problem, nseg: int = 1) -> int:
    return int(lib().gdn_workspace_bytes(ctypes.byref(prob), nseg))


def segmented_pieces(prob: Problem, nseg: int = 1) -> int:
    """Pieces per sequence the segmented forward uses on the current device (0: invalid)."""
    return int(lib().gdn_segmented_pieces(ctypes.byref(prob), nseg))


def segmented_plan(prob: Problem, nseg: int = 1):
    """(P, chunks of piece 0, chunks of each later piece) of the segmented forward's piece plan
    on the current device ((0, 0, 0): invalid)."""
    first, rest = ctypes.c_int(0), ctypes.c_int(0)
    P = lib().gdn_segmented_plan(ctypes.byref(prob), nseg, ctypes.byref(first), ctypes.byref(rest))
    return int(P), int(first.value), int(rest.value)


def alloc_workspace(prob: Problem, nseg: int = 1, device="cuda"):
    """A zeroed workspace tensor of the size the library asks for (torch owns the memory)."""
    import torch
    n = workspace_bytes(prob, nseg)
    if n == 0:
        raise GdnError(2, "gdn_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gdn_chunk_fwd(q, k, v, g, beta, h0, o, h_final, workspace, stream=None, prob=None):
    prob = prob or problem(k, v, o, g=g)
    _check(lib().gdn_chunk_fwd(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(h0), _ptr(o), _ptr(h_final), _ptr(workspace),
                               workspace.numel() if workspace is not None else 0,
                               _stream(stream)), "gdn_chunk_fwd")


def gdn_segment_summary(k, v, g, beta, M, S, nseg, workspace, stream=None, prob=None):
    prob = prob or problem(k, v, g=g)
    _check(lib().gdn_segment_summary(ctypes.byref(prob), nseg, _ptr(k), _ptr(v), _ptr(g),
                                     _ptr(beta), _ptr(M), _ptr(S), _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0,
                                     _stream(stream)), "gdn_segment_summary")


def gdn_summary_scan(M, S, h0, H_in, stream=None, prob=None):
    nseg, B, H, K, V = H_in.shape
    prob = prob or Problem(B, 0, H, K, V, 64, GDN_DTYPE_F32, GDN_DTYPE_F32)
    _check(lib().gdn_summary_scan(ctypes.byref(prob), nseg, _ptr(M), _ptr(S), _ptr(h0),
                                  _ptr(H_in), _stream(stream)), "gdn_summary_scan")


def gdn_segment_fwd(q, k, v, g, beta, H_in, o, h_final, nseg, workspace, stream=None,
                    prob=None):
    """The chunked forward of each of nseg segments from H_in[s] (None: zero states);
    workspace sized by workspace_bytes(prob, 1)."""
    prob = prob or problem(k, v, o, g=g)
    _check(lib().gdn_segment_fwd(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(beta), _ptr(H_in), _ptr(o), _ptr(h_final), _ptr(workspace),
                                 workspace.numel() if workspace is not None else 0,
                                 _stream(stream)), "gdn_segment_fwd")


def gdn_segmented_fwd(q, k, v, g, beta, h0, o, h_final, nseg, workspace, H_in=None,
                      stream=None, prob=None):
    prob = prob or problem(k, v, o, g=g)
    _check(lib().gdn_segmented_fwd(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(h_final),
                                   _ptr(H_in), _ptr(workspace),
                                   workspace.numel() if workspace is not None else 0,
                                   _stream(stream)), "gdn_segmented_fwd")


def gdn_segmented_fwd_timed(q, k, v, g, beta, h0, o, h_final, nseg, workspace, events,
                            H_in=None, stream=None, prob=None):
    """gdn_segmented_fwd recording five torch.cuda.Event (enable_timing=True) around its
    four stages: before the WY factors, before the first phase (piece 0's forward beside the
    piece summaries), before the scan, before the second phase (the forward of pieces
    1..P-1), after it."""
    prob = prob or problem(k, v, o, g=g)
    if len(events) != 5:
        raise ValueError("gdn_segmented_fwd_timed takes five events")
    arr = (_P * 5)(*[e.cuda_event for e in events])
    _check(lib().gdn_segmented_fwd_timed(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                         _ptr(h_final), _ptr(H_in), _ptr(workspace),
                                         workspace.numel() if workspace is not None else 0,
                                         _stream(stream), arr), "gdn_segmented_fwd_timed")


def gdn_segmented_fwd_noalloc(q, k, v, g, beta, h0, o, h_final, nseg, device_error=None,
                              stream=None, prob=None):
    """gdn_segmented_fwd with the library's fixed scratch array instead of a workspace.
    device_error: optional int32/uint32 CUDA tensor of >= 2 elements that receives the
    call's device error word {code, detail}."""
    prob = prob or problem(k, v, o, g=g)
    _check(lib().gdn_segmented_fwd_noalloc(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                           _ptr(h_final), _ptr(device_error), _stream(stream)),
           "gdn_segmented_fwd_noalloc")


def varlen_workspace_bytes(prob: Problem, nseq: int) -> int:
    return int(lib().gdn_varlen_workspace_bytes(ctypes.byref(prob), nseq))


def alloc_varlen_workspace(prob: Problem, nseq: int, device="cuda"):
    """A zeroed workspace tensor for gdn_varlen_fwd (torch owns the memory)."""
    import torch
    n = varlen_workspace_bytes(prob, nseq)
    if n == 0:
        raise GdnError(2, "gdn_varlen_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gdn_varlen_fwd(q, k, v, g, beta, h0, o, h_final, cu_seqlens, workspace, stream=None,
                   prob=None):
    """Packed variable-length forward: q, k, v, g, beta, o hold [1, T, H, *] tokens of
    nseq = len(cu_seqlens) - 1 sequences; cu_seqlens is an int32 CUDA tensor; h0 and h_final
    are [nseq, H, K, V] fp32 (or None)."""
    prob = prob or problem(k, v, o, g=g)
    nseq = int(cu_seqlens.numel()) - 1
    _check(lib().gdn_varlen_fwd(ctypes.byref(prob), nseq, _ptr(cu_seqlens), _ptr(q), _ptr(k),
                                _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(h_final),
                                _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                _stream(stream)), "gdn_varlen_fwd")


def gdn_varlen_fwd_timed(q, k, v, g, beta, h0, o, h_final, cu_seqlens, workspace, events,
                         stream=None, prob=None):
    """gdn_varlen_fwd recording five torch.cuda.Event (enable_timing=True): before the length
    check, the plan and the WY factors; before the first phase (the whole forward when no
    sequence is cut); before the scan; before the second phase; after it."""
    prob = prob or problem(k, v, o, g=g)
    if len(events) != 5:
        raise ValueError("gdn_varlen_fwd_timed takes five events")
    arr = (_P * 5)(*[e.cuda_event for e in events])
    nseq = int(cu_seqlens.numel()) - 1
    _check(lib().gdn_varlen_fwd_timed(ctypes.byref(prob), nseq, _ptr(cu_seqlens), _ptr(q),
                                      _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                      _ptr(h_final), _ptr(workspace),
                                      workspace.numel() if workspace is not None else 0,
                                      _stream(stream), arr), "gdn_varlen_fwd_timed")


def gdn_state_grad_summary(q, k, g, beta, dO, dS, nseg, dH_end=None, stream=None, prob=None):
    """Per-segment state gradients: dS [nseg,B,H,K,V] fp32 receives the gradient on the state
    entering each segment of its outputs' loss (sum dO . o) plus <dH_end[s], state leaving
    it> (dH_end None = 0). dO carries the output dtype (fp32 or bf16)."""
    prob = prob or problem(k, dO, dO, g=g)   # a [B,T,H,K] g sets gate_k: rejected below
    _check(lib().gdn_state_grad_summary(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(g),
                                        _ptr(beta), _ptr(dO), _ptr(dH_end), _ptr(dS),
                                        _stream(stream)), "gdn_state_grad_summary")


def gdn_state_grad_scan(M, dS, dht, dH_in, stream=None, prob=None):
    """Reverse scan: dH_in[s] = M[s]^T dH_in[s+1] + dS[s] with dH_in[nseg] = dht (None = 0)."""
    nseg, B, H, K, V = dH_in.shape
    prob = prob or Problem(B, 0, H, K, V, 64, GDN_DTYPE_F32, GDN_DTYPE_F32)
    _check(lib().gdn_state_grad_scan(ctypes.byref(prob), nseg, _ptr(M), _ptr(dS), _ptr(dht),
                                     _ptr(dH_in), _stream(stream)), "gdn_state_grad_scan")


def chunk_bwd_workspace_bytes(prob: Problem, nseg: int = 1) -> int:
    return int(lib().gdn_chunk_bwd_workspace_bytes(ctypes.byref(prob), nseg))


def alloc_bwd_workspace(prob: Problem, nseg: int = 1, device="cuda"):
    """A zeroed workspace tensor for gdn_chunk_bwd (torch owns the memory)."""
    import torch
    n = chunk_bwd_workspace_bytes(prob, nseg)
    if n == 0:
        raise GdnError(2, "gdn_chunk_bwd_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gdn_chunk_bwd(q, k, v, g, beta, h0, dO, dht, dq, dk, dv, dg, dbeta, dh0, nseg, workspace,
                  stream=None, prob=None):
    """The backward: fp32 gradients dq, dk [B,T,H,K], dv [B,T,H,V], dg, dbeta [B,T,H] and dh0
    [B,H,K,V] (None skips it) of sum(dO . o) + <dht, h_final>; dO has the output dtype, dht
    (fp32, or None) the state's shape."""
    prob = prob or problem(k, v, dO, g=g)
    _check(lib().gdn_chunk_bwd(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dht), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0), _ptr(workspace),
                               workspace.numel() if workspace is not None else 0,
                               _stream(stream)), "gdn_chunk_bwd")


def gdn_chunk_bwd_timed(q, k, v, g, beta, h0, dO, dht, dq, dk, dv, dg, dbeta, dh0, nseg,
                        workspace, events, stream=None, prob=None):
    """gdn_chunk_bwd with six torch.cuda.Event markers recorded between its steps."""
    if len(events) != 6:
        raise ValueError("gdn_chunk_bwd_timed takes six events")
    prob = prob or problem(k, v, dO, g=g)
    arr = (_P * 6)(*[e.cuda_event for e in events])
    _check(lib().gdn_chunk_bwd_timed(ctypes.byref(prob), nseg, _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(g), _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dht),
                                     _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta),
                                     _ptr(dh0), _ptr(workspace),
                                     workspace.numel() if workspace is not None else 0,
                                     _stream(stream), arr), "gdn_chunk_bwd_timed")


def _on_device(*tensors):
    """Raises ValueError unless every tensor (or None) lies contiguous on the current CUDA device:
    the library takes plain pointers and launches on that device."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    for i, t in enumerate(tensors):
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            if t.get_device() != dev:
                raise ValueError(f"tensor argument {i} is on {t.device}, not on the current CUDA device")
            raise ValueError(f"tensor argument {i} is not contiguous")


def _all_on(*tensors):
    """_on_device, in few steps; the current CUDA device."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            _on_device(*tensors)   # names what is wrong
    return dev


def _stream_on(stream, dev):
    """_stream on a device that is known to be the current one."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if stream is None and raw else _stream(stream)


def _is(name, t, dtype, shape):
    """Raises ValueError unless t (or None) has this dtype and shape."""
    if t is not None and (t.dtype is not dtype or t.shape != shape):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, not {dtype} {tuple(shape)}")


def alloc_recurrent_workspace(num_slots: int, device="cuda"):
    """A zeroed workspace tensor for gdn_recurrent_fwd on a cache of num_slots slots."""
    import torch
    n = int(lib().gdn_recurrent_workspace_bytes(num_slots))
    if n == 0:
        raise GdnError(1, "gdn_recurrent_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gdn_recurrent_fwd(q, k, v, g, beta, state, slots_in, slots_out, o, workspace, cu_seqlens=None,
                      per_token=False, decay_first=False, stream=None):
    """The rule token by token over a state cache [num_slots, H, K, V] fp32: q, k [B, T, Hqk, K],
    v, o [B, T, H, V], g [B, T, H] (or [B, T, H, K]), beta [B, T, H]. Without cu_seqlens B
    sequences of T tokens; with it (int32, on the GPU) B == 1 and len(cu_seqlens) - 1 packed
    sequences. slots_in, slots_out: int32 GPU tensors (or None), one entry a sequence; with
    per_token slots_out has one entry a token. Negative entries: a zero state, not written."""
    import torch
    vshape, kshape, dt = v.shape, k.shape, k.dtype
    B, T, H, V = vshape
    _, _, Hqk, K = kshape
    nseq = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _on_device(q, k, v, g, beta, state, slots_in, slots_out, o, workspace, cu_seqlens)
    gate_k = g.dim() == 4
    slots = 0 if state is None else state.shape[0]
    want = (("q", q, dt, kshape), ("v", v, dt, (B, T, H, V)), ("o", o, o.dtype, vshape),
            ("g", g, dt, (B, T, H, K) if gate_k else (B, T, H)), ("beta", beta, dt, (B, T, H)),
            ("state", state, torch.float32, (slots, H, K, V)), ("slots_in", slots_in, torch.int32, (nseq,)),
            ("slots_out", slots_out, torch.int32, (B * T if per_token else nseq,)),
            ("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,)))
    for name, t, dtype, shape in want:
        if t is not None and (t.dtype is not dtype or t.shape != shape):
            _is(name, t, dtype, shape)   # names what is wrong
    if kshape[:2] != (B, T):
        raise ValueError(f"k is {tuple(kshape)}, v {tuple(vshape)}")
    prob = Problem(B, T, H, K, V, 64, _dtype_code(k), _dtype_code(o), decay_first, gate_k)
    _check(lib().gdn_recurrent_fwd(ctypes.byref(prob), Hqk, nseq, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(),
                                   v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(state), slots,
                                   _ptr(slots_in), _ptr(slots_out), per_token, o.data_ptr(), *_room(workspace),
                                   _stream(stream)), "gdn_recurrent_fwd")


def alloc_cache_workspace(num_pages: int, n: int = 0, device="cuda"):
    """A zeroed workspace tensor for the gdn_cache calls on a cache of num_pages pages, with at most
    n pairs (copy) or requests (fork) a call."""
    import torch
    size = int(lib().gdn_cache_workspace_bytes(num_pages, n))
    if size == 0:
        raise GdnError(1, "gdn_cache_workspace_bytes")
    return torch.zeros(size, dtype=torch.uint8, device=device)


def _int(name, n):
    """n, which the library takes as a C int (ctypes would cut it off without a word)."""
    if n >= 2**31:
        raise ValueError(f"{name} is {n}, more than the library counts to")
    return n


def _pages(pages):
    if pages.dim() < 3:
        raise ValueError("pages is [layers, num_pages, ...]")
    layers, num = _int("the number of layers", pages.shape[0]), _int("the number of pages", pages.shape[1])
    total = pages.numel() * pages.element_size()
    return pages.data_ptr(), layers, num, total // (layers * num) if total else 0


def _indexes(**arrays):
    """Lengths aside, index arrays are one-dimensional int32."""
    import torch
    for name, t in arrays.items():
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1):
            raise ValueError(f"{name} is not a one-dimensional int32 tensor")
        if t is not None:
            _int(f"the length of {name}", t.numel())


def _room(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def gdn_cache_copy(pages, src, dst, workspace, stream=None):
    """pages [layers, num_pages, ...]: page dst[i] := page src[i] in every layer (zeros for a
    negative src, nothing for a negative dst); src, dst int32 GPU tensors."""
    _on_device(pages, src, dst, workspace)
    _indexes(src=src, dst=dst)
    if src.numel() != dst.numel():
        raise ValueError("src and dst differ in length")
    _check(lib().gdn_cache_copy(*_pages(pages), src.numel(), _ptr(src), _ptr(dst), *_room(workspace),
                                _stream(stream)), "gdn_cache_copy")


def gdn_cache_fork(pages, refs, parents, children, workspace, share=False, stream=None):
    """A copy of page parents[i] (zeros for a negative one) in the next of the lowest-numbered free
    pages (refs 0), its number in children[i] (-1: refused); share: the parent gains a user
    instead. refs, parents, children int32 GPU tensors."""
    _on_device(pages, refs, parents, children, workspace)
    _indexes(refs=refs, parents=parents, children=children)
    if parents.numel() != children.numel() or refs.numel() != pages.shape[1]:
        raise ValueError("one child a parent and one count a page are wanted")
    _check(lib().gdn_cache_fork(*_pages(pages), _ptr(refs), parents.numel(), _ptr(parents),
                                _ptr(children), int(share), *_room(workspace), _stream(stream)),
           "gdn_cache_fork")


def gdn_cache_free(refs, pages, workspace, stream=None):
    """One user less of every page named in `pages` (int32; negative entries are skipped)."""
    _on_device(refs, pages, workspace)
    _indexes(refs=refs, pages=pages)
    _check(lib().gdn_cache_free(refs.numel(), _ptr(refs), pages.numel(), _ptr(pages),
                                *_room(workspace), _stream(stream)), "gdn_cache_free")


def gdn_cache_compact(pages, refs, table, remap, live, workspace, stream=None):
    """The pages in use move to the front of the cache; table (or None) is rewritten to the new
    numbers, remap [num_pages] (or None) and live [1] (or None) receive every page's new number
    and how many are in use."""
    _on_device(pages, refs, table, remap, live, workspace)
    _indexes(refs=refs, table=table, remap=remap, live=live)
    num = pages.shape[1]
    if refs.numel() != num or (remap is not None and remap.numel() != num) or (
            live is not None and live.numel() != 1):
        raise ValueError("one count and one new number a page are wanted, and one int for live")
    _check(lib().gdn_cache_compact(*_pages(pages), _ptr(refs), 0 if table is None else table.numel(),
                                   _ptr(table), _ptr(remap), _ptr(live), *_room(workspace),
                                   _stream(stream)), "gdn_cache_compact")


def _rows(x, y_like, params, **rest):
    """(rows, N) of x [..., N]; the tensors of y's type have x's shape, the parameters are fp32 [N]."""
    import torch
    N = _int("the length of a row", x.shape[-1])
    for name, t in rest.items():
        _is(name, t, y_like.dtype, x.shape)
    for name, t in params.items():
        _is(name, t, torch.float32, (N,))
    return x.numel() // N if N else 0, N


def gdn_norm_fwd(x, w, b, z, y, eps=1e-6, rms=True, stream=None):
    """y = ((x - m) s w + b) z sigmoid(z) row by row: x, z, y [..., N], w, b [N] fp32 (w, b, z may
    be None); rms: the root-mean-square norm (m = 0), else the layer norm. z has y's type."""
    _on_device(x, w, b, z, y)
    rows, N = _rows(x, y, dict(w=w, b=b), z=z, y=y)
    _check(lib().gdn_norm_fwd(rows, N, _dtype_code(x), _dtype_code(y), int(rms), eps, _ptr(x), _ptr(w),
                              _ptr(b), _ptr(z), _ptr(y), _stream(stream)), "gdn_norm_fwd")


def alloc_norm_bwd_workspace(rows: int, N: int, device="cuda"):
    """A workspace tensor for gdn_norm_bwd on rows rows of N values."""
    import torch
    n = int(lib().gdn_norm_bwd_workspace_bytes(rows, N))
    if n == 0:
        raise GdnError(2, "gdn_norm_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def gdn_norm_bwd(x, w, b, z, dy, dx, dz, dw, db, workspace, eps=1e-6, rms=True, stream=None):
    """Gradients of gdn_norm_fwd for dy (z's and y's type): dx (x's type), dz (None skips it), dw, db
    [N] fp32 (None skips either)."""
    _on_device(x, w, b, z, dy, dx, dz, dw, db, workspace)
    rows, N = _rows(x, dy, dict(w=w, b=b, dw=dw, db=db), z=z, dy=dy, dz=dz)
    _is("dx", dx, x.dtype, x.shape)
    _check(lib().gdn_norm_bwd(rows, N, _dtype_code(x), _dtype_code(dy), int(rms), eps, _ptr(x), _ptr(w),
                              _ptr(b), _ptr(z), _ptr(dy), _ptr(dx), _ptr(dz), _ptr(dw), _ptr(db),
                              *_room(workspace), _stream(stream)), "gdn_norm_bwd")


def _linear(q, k, v, decay, o, cu_seqlens, states, **more):
    """(problem, Hqk, nseq) of a linear-attention call, its tensors' shapes and types checked: q, k [B, T, Hqk, K], v
    and what is like it [B, T, H, V], states [nseq, H, K, V] fp32, o (or its gradient) of a type of its own."""
    import torch
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError(f"k is {tuple(k.shape)}, v {tuple(v.shape)}, not [B, T, heads, channels]")
    B, T, H, V = v.shape
    Hqk, K = k.shape[2:]
    nseq = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if k.shape[:2] != (B, T):
        raise ValueError(f"k is {tuple(k.shape)}, v {tuple(v.shape)}")
    for name, n in (("B", B), ("T", T), ("H", H), ("the number of sequences", nseq)):
        _int(name, n)
    _is("q", q, k.dtype, k.shape)
    _is("v", v, k.dtype, v.shape)
    _is("o", o, None if o is None else o.dtype, v.shape)
    _is("decay", decay, torch.float32, (H,))
    _is("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,))
    for name, t in states.items():
        _is(name, t, torch.float32, (nseq, H, K, V))
    for name, (t, like) in more.items():
        _is(name, t, like.dtype, like.shape)
    return Problem(B, T, H, K, V, 64, _dtype_code(k), _dtype_code(v if o is None else o), 0, 0), Hqk, nseq


def alloc_linear_workspace(k, v, cu_seqlens=None, backward=False):
    """A zeroed workspace tensor for gdn_linear_fwd (or gdn_linear_bwd) on tensors of these shapes, on their device."""
    import torch
    prob, Hqk, nseq = _linear(k, k, v, None, None, cu_seqlens, {})
    n = int(lib().gdn_linear_workspace_bytes(ctypes.byref(prob), Hqk, nseq, int(backward)))
    if n == 0:
        raise GdnError(2, "gdn_linear_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=k.device)


@functools.lru_cache(maxsize=256)
def _linear_problem(vshape, kshape, nseq, in_dtype, out_dtype):
    """The problem of these shapes and types, or None where they do not fit together (their tensors are then looked at one
    by one). Kept, so that a call of known sizes costs the host little: it is read only."""
    if len(vshape) != 4 or len(kshape) != 4 or kshape[:2] != vshape[:2] or max(*vshape, *kshape, nseq) >= 2**31:
        return None
    return Problem(*vshape[:3], kshape[3], vshape[3], 64, _CODES[in_dtype], _CODES[out_dtype], 0, 0)


def _linear_call(q, k, v, decay, o, cu_seqlens, kv, states, dev):
    """(problem, nseq) of a call whose tensors fit: kv are those of k's and v's shapes, states those of the states'; else
    ValueError. As _linear, in few steps."""
    import torch
    vshape, kshape, dt, f32 = v.shape, k.shape, k.dtype, torch.float32
    nseq = vshape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    prob = _linear_problem(vshape, kshape, nseq, dt, o.dtype)
    ok = (prob is not None and q.dtype is dt and v.dtype is dt and q.shape == kshape and o.shape == vshape and
          decay is not None and decay.dtype is f32 and decay.shape == vshape[2:3] and
          (cu_seqlens is None or (cu_seqlens.dtype is torch.int32 and cu_seqlens.dim() == 1)))
    if ok:
        for t, shape in kv:
            ok = ok and t.dtype is dt and t.shape == shape
        want = (nseq, vshape[2], kshape[3], vshape[3])
        for t in states:
            ok = ok and (t is None or (t.dtype is f32 and t.shape == want))
    return (prob if ok else None), nseq


def gdn_linear_fwd(q, k, v, decay, h0, o, h_final, workspace, cu_seqlens=None, stream=None):
    """Linear attention with a decay for each head, H_t = exp(decay[h]) H_{t-1} + k_t v_t^T, o_t = q_t^T H_t, in chunks: q, k
    [B, T, Hqk, K], v, o [B, T, H, V], decay [H] fp32, h0, h_final [nseq, H, K, V] fp32 (or None). Without cu_seqlens B
    sequences of T tokens; with it (int32, on the GPU) B == 1 and len(cu_seqlens) - 1 packed sequences."""
    dev = _all_on(q, k, v, decay, h0, o, h_final, workspace, cu_seqlens)
    prob, nseq = _linear_call(q, k, v, decay, o, cu_seqlens, (), (h0, h_final), dev)
    if prob is None:
        prob, _, nseq = _linear(q, k, v, decay, o, cu_seqlens, dict(h0=h0, h_final=h_final))
    _check(lib().gdn_linear_fwd(prob, k.shape[2], nseq, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                _ptr(decay), _ptr(h0), o.data_ptr(), _ptr(h_final), *_room(workspace),
                                _stream_on(stream, dev)), "gdn_linear_fwd")


def gdn_linear_bwd(q, k, v, decay, h0, dO, dht, dq, dk, dv, dh0, workspace, cu_seqlens=None, stream=None):
    """Gradients of gdn_linear_fwd for dO (o's type) and dht (or None): dq, dk, dv (q's, k's and v's shape and type) and
    dh0 (or None). workspace: alloc_linear_workspace(..., backward=True)."""
    dev = _all_on(q, k, v, decay, h0, dO, dht, dq, dk, dv, dh0, workspace, cu_seqlens)
    prob, nseq = _linear_call(q, k, v, decay, dO, cu_seqlens, ((dq, k.shape), (dk, k.shape), (dv, v.shape)), (h0, dht, dh0), dev)
    if prob is None:
        prob, _, nseq = _linear(q, k, v, decay, dO, cu_seqlens, dict(h0=h0, dht=dht, dh0=dh0), dq=(dq, q), dk=(dk, k),
                                dv=(dv, v))
    _check(lib().gdn_linear_bwd(prob, k.shape[2], nseq, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                _ptr(decay), _ptr(h0), dO.data_ptr(), _ptr(dht), dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), _ptr(dh0), *_room(workspace), _stream_on(stream, dev)), "gdn_linear_bwd")


def gdn_linear_recurrent_fwd(q, k, v, decay, state, slots_in, slots_out, o, workspace, cu_seqlens=None,
                             per_token=False, stream=None):
    """The same rule token by token over a state cache [num_slots, H, K, V] fp32, as gdn_recurrent_fwd takes it;
    workspace: alloc_recurrent_workspace(num_slots)."""
    import torch
    dev = _all_on(q, k, v, decay, state, slots_in, slots_out, o, workspace, cu_seqlens)
    prob, nseq = _linear_call(q, k, v, decay, o, cu_seqlens, (), (), dev)
    if prob is None:
        prob, _, nseq = _linear(q, k, v, decay, o, cu_seqlens, {})
    vshape, slots = v.shape, 0
    if state is not None:
        slots = state.shape[0]
        if slots >= 2**31 or state.dtype is not torch.float32 or state.shape[1:] != (vshape[2], k.shape[3], vshape[3]):
            _is("state", state, torch.float32, (_int("the number of slots", slots), vshape[2], k.shape[3], vshape[3]))
    for name, t, n in (("slots_in", slots_in, nseq), ("slots_out", slots_out, vshape[0] * vshape[1] if per_token else nseq)):
        if t is not None and (t.dtype is not torch.int32 or t.shape != (n,)):
            _is(name, t, torch.int32, (n,))
    _check(lib().gdn_linear_recurrent_fwd(prob, k.shape[2], nseq, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                          _ptr(decay), _ptr(state), slots, _ptr(slots_in), _ptr(slots_out),
                                          per_token, o.data_ptr(), *_room(workspace), _stream_on(stream, dev)),
           "gdn_linear_recurrent_fwd")


def _head_stride(name, t, like=None):
    """Values from one token of t [B, T, heads, K] to the next; within a token the heads lie side by side."""
    if t.dim() != 4:
        raise ValueError(f"{name} is {tuple(t.shape)}, not [B, T, heads, K]")
    B, T, H, K = t.shape
    if like is not None:
        _is(name, t, like.dtype, like.shape)
    b, n, h, c = t.stride()
    n = n if T > 1 else b if B > 1 else H * K    # (the strides of axes of one entry say nothing)
    if (c != 1 and K > 1) or (h != K and H > 1) or (B > 1 and T > 1 and b != T * n) or n < H * K:
        raise ValueError(f"{name} has strides {t.stride()}: wanted are heads side by side, tokens evenly apart")
    return n


@functools.lru_cache(maxsize=256)
def _qk_problem(qshape, Hk, R, interleaved, x_dtype, y_dtype, eps, q_stride, k_stride):
    return QkProblem(*qshape[:3], Hk, qshape[3], R, interleaved, _CODES[x_dtype], _CODES[y_dtype], eps, q_stride, k_stride)


def _qk(q, k, wq, wk, freq, yq, yk, positions, eps, interleaved, dev):
    """The problem of these heads; yq, yk are contiguous and of one type."""
    import torch
    f32, qshape, kshape = torch.float32, q.shape, k.shape
    if q.get_device() != dev or k.get_device() != dev:
        name, t = ("q", q) if q.get_device() != dev else ("k", k)
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    qs = qshape[2] * qshape[3] if len(qshape) == 4 and q.is_contiguous() else _head_stride("q", q)
    ks = kshape[2] * kshape[3] if len(kshape) == 4 and k.is_contiguous() else _head_stride("k", k)
    B, T, Hq, K = qshape
    if max(qshape) >= 2**31 or kshape[2] >= 2**31:
        for name, n in (("B", B), ("T", T), ("Hq", Hq), ("Hk", kshape[2]), ("K", K)):
            _int(name, n)
    R = 0 if freq is None else 2 * freq.numel()
    for name, t, dtype, shape in (("k", k, q.dtype, (B, T, kshape[2], K)), ("wq", wq, f32, (K,)), ("wk", wk, f32, (K,)),
                                  ("freq", freq, f32, (R // 2,)), ("the queries' results", yq, yq.dtype, qshape),
                                  ("the keys' results", yk, yq.dtype, kshape)):
        if t is not None and (t.dtype is not dtype or t.shape != shape):
            _is(name, t, dtype, shape)
    if positions is not None and (positions.dtype is not torch.int32 or positions.numel() != B * T):
        raise ValueError("positions holds one int32 a token")
    return _qk_problem(qshape, kshape[2], R, int(interleaved), q.dtype, yq.dtype, eps, qs, ks)


def gdn_qk_norm_fwd(q, k, wq, wk, freq, yq, yk, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Every head of q [B, T, Hq, K] and k [B, T, Hk, K] (tokens evenly apart: parts of one projection's rows, say)
    normalised by its root mean square, scaled by wq, wk [K] fp32 (or None) and rotated by its position: freq [R / 2]
    fp32 (or None: not rotated), positions int32 (or None: 0 .. T - 1). yq, yk: contiguous, of one type."""
    dev = _all_on(wq, wk, freq, positions, yq, yk)
    prob = _qk(q, k, wq, wk, freq, yq, yk, positions, eps, interleaved, dev)
    _check(lib().gdn_qk_norm_fwd(prob, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(freq), _ptr(positions),
                                 yq.data_ptr(), yk.data_ptr(), _stream_on(stream, dev)), "gdn_qk_norm_fwd")


def alloc_qk_norm_bwd_workspace(q, k=None):
    """A workspace tensor for gdn_qk_norm_bwd on heads like q's, on its device."""
    import torch
    n = int(lib().gdn_qk_norm_bwd_workspace_bytes(_int("K", q.shape[-1])))
    if n == 0:
        raise GdnError(2, "gdn_qk_norm_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def gdn_qk_norm_bwd(q, k, wq, wk, freq, dyq, dyk, dq, dk, dwq, dwk, workspace, positions=None, eps=1e-6,
                    interleaved=False, stream=None):
    """Gradients of gdn_qk_norm_fwd for dyq, dyk (contiguous): dq, dk (q's and k's type, shape and token stride), dwq, dwk [K]
    fp32 (None skips either)."""
    import torch
    dev = _all_on(wq, wk, freq, positions, dyq, dyk, dwq, dwk, workspace)
    prob = _qk(q, k, wq, wk, freq, dyq, dyk, positions, eps, interleaved, dev)
    for name, t, like, stride in (("dq", dq, q, prob.q_stride), ("dk", dk, k, prob.k_stride)):
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
        if _head_stride(name, t, like) != stride and t.shape[0] * t.shape[1] > 1:
            raise ValueError(f"{name} has another token stride than its input")
    K = q.shape[-1]
    _is("dwq", dwq, torch.float32, (K,))
    _is("dwk", dwk, torch.float32, (K,))
    _check(lib().gdn_qk_norm_bwd(prob, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(freq), _ptr(positions),
                                 dyq.data_ptr(), dyk.data_ptr(), dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk),
                                 *_room(workspace), _stream_on(stream, dev)), "gdn_qk_norm_bwd")


def gdn_selftest_wait_timeout(workspace, limit_cycles, stream=None):
    """Launches the bounded-wait self-test (a wait that runs out after limit_cycles SM cycles
    and records GDN_ERR_TIMEOUT in the workspace's error word); read it with
    gdn_check_device_error."""
    _check(lib().gdn_selftest_wait_timeout(_ptr(workspace), int(limit_cycles), _stream(stream)),
           "gdn_selftest_wait_timeout")


def gdn_check_device_error(workspace, stream=None):
    """Synchronises, returns (status, detail) from the workspace's device error word."""
    detail = ctypes.c_uint(0)
    st = lib().gdn_check_device_error(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)
