"""Causal flash attention on one NVIDIA GB300 (sm_103a): thin Python binding of
libfa (include/fa.h).

The functions with the C names (`fa_fwd`, `fa_bwd`, `fa_bwd_workspace_bytes`,
`fa_fwd_kv`, `fa_bwd_kv`, `fa_bwd_kv_workspace_bytes`, `fa_fwd_splitkv`,
`fa_fwd_splitkv_workspace_bytes`, `fa_fwd_splitkv_paged`, `fa_strerror`,
`fa_last_device_status`, `fa_version`) only marshal arguments:
shapes come from the tensors, pointers from `data_ptr()`, and the stream from
PyTorch's current stream. Every step of the computation runs in libfa's CUDA
kernels; there is no other code path. `attention_forward` / `attention_backward`
additionally allocate their outputs (and the backward workspace) with
PyTorch.

The calls for span attention, the ragged paged cache and query/key preparation
go through a native module beside the library (_fa_torch, csrc/fa_torch.cpp), which
checks the tensors, allocates what is missing and makes the library call: one of
them is a few microseconds of host time.

Library and module are built in-tree by `causal_flash_attention_gb300.build.build()`;
loading them raises if they have not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import torch

__all__ = [
    "FAError", "lib", "fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_strerror",
    "fa_last_device_status", "fa_version", "attention_forward", "attention_backward",
    "DTYPE_CODES", "fa_bwd_noalloc", "NOALLOC_SCRATCH_BYTES", "fa_fwd_kv", "fa_bwd_kv",
    "fa_bwd_kv_workspace_bytes", "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_bytes",
    "decode_forward", "fa_fwd_splitkv_paged", "decode_forward_paged",
    "fa_fwd_span", "fa_bwd_span", "fa_bwd_span_workspace_bytes", "attention_span_forward",
    "attention_span_backward", "key_spans", "fa_fwd_ragged_paged",
    "fa_fwd_ragged_paged_workspace_bytes", "decode_forward_ragged", "fa_qk_norm_rope",
    "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_bytes", "fa_qk_norm_rope_append",
    "qk_norm_rope_forward", "qk_norm_rope_backward", "qk_norm_rope_append", "rope_inv_freq",
    "rope_turns", "decode_step_ragged",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")
DTYPE_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_lib = None


class _View(ctypes.Structure):
    """fa_view: a strided [B, H, S, d] tensor whose last dimension is contiguous."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong), ("stride_s", ctypes.c_longlong)]


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {fa_strerror(code)} (code {code})")


def lib() -> ctypes.CDLL:
    """Load libfa.so (once) and declare its C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with causal_flash_attention_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp]
    L.fa_fwd.restype = i32
    L.fa_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.fa_bwd_workspace_bytes.restype = sz
    L.fa_bwd.argtypes = [vp] * 9 + [i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
    L.fa_bwd.restype = i32
    L.fa_fwd_kv.argtypes = [vp, vp, vp, vp, vp] + [i32] * 7 + [f32, i32, vp]
    L.fa_fwd_kv.restype = i32
    L.fa_bwd_kv_workspace_bytes.argtypes = [i32] * 6
    L.fa_bwd_kv_workspace_bytes.restype = sz
    L.fa_bwd_kv.argtypes = [vp] * 9 + [i32] * 7 + [f32, i32, vp, sz, vp]
    L.fa_bwd_kv.restype = i32
    L.fa_fwd_splitkv.argtypes = [vp] * 5 + [i32] * 7 + [f32, i32, i32, vp, sz, vp]
    L.fa_fwd_splitkv.restype = i32
    L.fa_fwd_splitkv_workspace_bytes.argtypes = [i32] * 7
    L.fa_fwd_splitkv_workspace_bytes.restype = sz
    L.fa_fwd_splitkv_paged.argtypes = [vp] * 6 + [i32] * 10 + [f32, i32, i32, vp, sz, vp]
    L.fa_fwd_splitkv_paged.restype = i32
    L.fa_fwd_span.argtypes = [vp] * 7 + [i32] * 6 + [f32, f32, vp, i32, vp]
    L.fa_fwd_span.restype = i32
    L.fa_bwd_span_workspace_bytes.argtypes = [i32] * 6
    L.fa_bwd_span_workspace_bytes.restype = sz
    L.fa_bwd_span.argtypes = [vp] * 11 + [i32] * 6 + [f32, f32, vp, i32, vp, sz, vp]
    L.fa_bwd_span.restype = i32
    L.fa_fwd_ragged_paged.argtypes = [vp] * 7 + [i32] * 9 + [f32, f32, vp, i32, vp, sz, vp]
    L.fa_fwd_ragged_paged.restype = i32
    L.fa_fwd_ragged_paged_workspace_bytes.argtypes = [i32] * 7
    L.fa_fwd_ragged_paged_workspace_bytes.restype = sz
    vw = ctypes.POINTER(_View)
    L.fa_qk_norm_rope.argtypes = [vw] * 4 + [vp, vp, f32, vp, vp, i32, i32, f32] + [i32] * 6 + [vp]
    L.fa_qk_norm_rope.restype = i32
    L.fa_qk_norm_rope_bwd.argtypes = ([vw] * 6 + [vp] * 4 + [f32, vp, vp, i32, i32, f32]
                                      + [i32] * 6 + [vp, sz, vp])
    L.fa_qk_norm_rope_bwd.restype = i32
    L.fa_qk_norm_rope_bwd_workspace_bytes.argtypes = [i32] * 6
    L.fa_qk_norm_rope_bwd_workspace_bytes.restype = sz
    L.fa_qk_norm_rope_append.argtypes = ([vw] * 4 + [vp] * 6 + [f32, vp, i32, i32, f32]
                                         + [i32] * 9 + [vp])
    L.fa_qk_norm_rope_append.restype = i32
    L.fa_strerror.argtypes = [i32]
    L.fa_strerror.restype = ctypes.c_char_p
    L.fa_last_device_status.argtypes = [vp, ctypes.POINTER(i32)]
    L.fa_last_device_status.restype = i32
    L.fa_version.argtypes = []
    L.fa_version.restype = i32
    _lib = L
    return L


def fa_strerror(code: int) -> str:
    return lib().fa_strerror(int(code)).decode()


def fa_version() -> int:
    return int(lib().fa_version())


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's raw handle straight from PyTorch's C layer, where the
# build has it (a cheap call; torch.cuda.current_stream() builds a Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_NULL_CONTEXT = contextlib.nullcontext()


def _stream(stream, t=None):
    """The CUDA stream handle for a call: `stream` itself, or PyTorch's current
    stream on t's device (the current device when t is None)."""
    if stream is None:
        if _raw_stream is not None and t is not None and t.is_cuda:
            return _raw_stream(t.get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dims(q, k):
    """(B, Hq, Hkv, S, d) of a self-attention call (q and k of one length)."""
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    if Sq != Skv:
        raise ValueError(f"q has {Sq} rows and k {Skv}: use the *_kv functions")
    return B, Hq, Hkv, Sq, d


def _dims_kv(q, k):
    """(B, Hq, Hkv, Sq, Skv, d) from q [B,Hq,Sq,d] and k [B,Hkv,Skv,d]."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, S, d]")
    B, Hq, Sq, d = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    return int(B), int(Hq), int(Hkv), int(Sq), int(Skv), int(d)


def _on_device(t):
    """Make t's GPU the current device for the call (the library runs on the
    current device); nothing to switch when it already is."""
    if t is not None and t.is_cuda and t.get_device() != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return _NULL_CONTEXT


def _check_contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def fa_fwd(q, k, v, out, lse, causal=True, scale=None, stream=None):
    """Call fa_fwd on caller-provided tensors (out: like q; lse: float32 [B,Hq,S])."""
    _check_contig(q, k, v, out, lse)
    B, Hq, Hkv, S, d = _dims(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    with _on_device(q):
        rc = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, S, d,
                          int(bool(causal)), scale, DTYPE_CODES.get(q.dtype, -1), _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_fwd")


def fa_bwd_workspace_bytes(B, Hq, Hkv, S, d) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Hq, Hkv, S, d))


def fa_bwd(q, k, v, out, dout, lse, dq, dk, dv, workspace, causal=True, scale=None,
           stream=None):
    """Call fa_bwd on caller-provided tensors; `workspace` is a device tensor of at
    least fa_bwd_workspace_bytes(...) bytes."""
    _check_contig(q, k, v, out, dout, lse, dq, dk, dv)
    B, Hq, Hkv, S, d = _dims(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(q):
        rc = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                          _ptr(dk), _ptr(dv), B, Hq, Hkv, S, d, int(bool(causal)), scale,
                          DTYPE_CODES.get(q.dtype, -1), _ptr(workspace), ws_bytes, _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_bwd")


def fa_fwd_kv(q, k, v, out, lse, causal=True, scale=None, stream=None):
    """Call fa_fwd_kv: q/out [B,Hq,Sq,d], k/v [B,Hkv,Skv,d], lse float32 [B,Hq,Sq];
    the causal mask is aligned to the last key (kv_offset = Skv - Sq)."""
    _check_contig(q, k, v, out, lse)
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    with _on_device(q):
        rc = lib().fa_fwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                             d, int(bool(causal)), scale, DTYPE_CODES.get(q.dtype, -1),
                             _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_fwd_kv")


def fa_bwd_kv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d) -> int:
    return int(lib().fa_bwd_kv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d))


def fa_bwd_kv(q, k, v, out, dout, lse, dq, dk, dv, workspace, causal=True, scale=None,
              stream=None):
    """Call fa_bwd_kv (separate query and key/value lengths, as fa_fwd_kv)."""
    _check_contig(q, k, v, out, dout, lse, dq, dk, dv)
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(q):
        rc = lib().fa_bwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, d, int(bool(causal)), scale,
                             DTYPE_CODES.get(q.dtype, -1), _ptr(workspace), ws_bytes,
                             _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_bwd_kv")


def fa_fwd_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d, n_splits=0) -> int:
    return int(lib().fa_fwd_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d, n_splits))


def fa_fwd_splitkv(q, k, v, out, lse, causal=True, scale=None, n_splits=0, workspace=None,
                   stream=None):
    """Call fa_fwd_splitkv (few query rows against a long key/value sequence);
    `workspace` is a device tensor of at least fa_fwd_splitkv_workspace_bytes(...)
    bytes, or None when that size is 0."""
    _check_contig(q, k, v, out, lse)
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(q):
        rc = lib().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq,
                                  Skv, d, int(bool(causal)), scale, DTYPE_CODES.get(q.dtype, -1),
                                  int(n_splits), _ptr(workspace), ws_bytes, _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_fwd_splitkv")


def decode_forward(q, k, v, causal=True, scale=None, n_splits=0, stream=None):
    """Allocate out, lse and the split workspace with PyTorch and run
    fa_fwd_splitkv. Returns (out, lse)."""
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    n = fa_fwd_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d, n_splits)
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    fa_fwd_splitkv(q, k, v, out, lse, causal, scale, n_splits, ws, stream)
    return out, lse


def fa_fwd_splitkv_paged(q, k_cache, v_cache, block_table, out, lse, Skv, causal=True,
                         scale=None, n_splits=0, workspace=None, stream=None):
    """Call fa_fwd_splitkv_paged: q [B,Hq,Sq,d]; k_cache/v_cache
    [num_blocks,Hkv,block_size,d]; block_table int32 [B,max_blocks]; every
    sequence holds Skv keys."""
    _check_contig(q, k_cache, v_cache, block_table, out, lse)
    if q.dim() != 4 or k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q [B,Hq,Sq,d], caches [num_blocks,Hkv,block_size,d], table [B,max_blocks]")
    if block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32")
    B, Hq, Sq, d = (int(x) for x in q.shape)
    num_blocks, Hkv, block_size = (int(x) for x in k_cache.shape[:3])
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on_device(q):
        rc = lib().fa_fwd_splitkv_paged(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(out), _ptr(lse), B, Hq,
            Hkv, Sq, int(Skv), d, block_size, num_blocks, int(block_table.shape[1]),
            int(bool(causal)), scale, DTYPE_CODES.get(q.dtype, -1), int(n_splits), _ptr(workspace),
            ws_bytes, _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_fwd_splitkv_paged")


def decode_forward_paged(q, k_cache, v_cache, block_table, Skv, causal=True, scale=None,
                         n_splits=0, stream=None):
    """Allocate out, lse and the split workspace and run fa_fwd_splitkv_paged."""
    B, Hq, Sq, d = (int(x) for x in q.shape)
    Hkv = int(k_cache.shape[1])
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    n = fa_fwd_splitkv_workspace_bytes(B, Hq, Hkv, Sq, int(Skv), d, n_splits)
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    fa_fwd_splitkv_paged(q, k_cache, v_cache, block_table, out, lse, Skv, causal, scale, n_splits,
                         ws, stream)
    return out, lse


def fa_last_device_status(stream=None) -> int:
    st = ctypes.c_int(0)
    rc = lib().fa_last_device_status(_stream(stream), ctypes.byref(st))
    if rc != 0:
        raise FAError(rc, "fa_last_device_status")
    return st.value


def attention_forward(q, k, v, causal=True, scale=None, stream=None):
    """Allocate out and lse with PyTorch and run fa_fwd (fa_fwd_kv when q and k
    have different lengths). Returns (out, lse)."""
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if q.shape[2] == k.shape[2]:
        fa_fwd(q, k, v, out, lse, causal, scale, stream)
    else:
        fa_fwd_kv(q, k, v, out, lse, causal, scale, stream)
    return out, lse


def workspace_for(q, k):
    B, Hq, Hkv, Sq, Skv, d = _dims_kv(q, k)
    n = fa_bwd_kv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attention_backward(q, k, v, out, dout, lse, causal=True, scale=None, workspace=None,
                       stream=None):
    """Allocate dq, dk, dv (and a workspace unless given) and run fa_bwd
    (fa_bwd_kv when q and k have different lengths)."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = workspace_for(q, k)
    if q.shape[2] == k.shape[2]:
        fa_bwd(q, k, v, out, dout, lse, dq, dk, dv, workspace, causal, scale, stream)
    else:
        fa_bwd_kv(q, k, v, out, dout, lse, dq, dk, dv, workspace, causal, scale, stream)
    return dq, dk, dv


# ------------------------------------------------------------- key spans --
_native_module = None


def _native():
    """The native part of the binding (loaded once)."""
    global _native_module
    if _native_module is None:
        try:
            from . import _fa_torch
        except ImportError as e:
            raise RuntimeError("the native binding module is missing: build it with "
                               "causal_flash_attention_gb300.build.build()") from e
        _native_module = _fa_torch
    return _native_module


def _call(name, where, *args, stream=None):
    """Call the native function `name` with the loaded library; FAError for the library's
    error codes, named after its entry point `where`."""
    if stream is not None and not isinstance(stream, int):
        stream = stream.cuda_stream
    r = getattr(_native_module or _native(), name)((_lib or lib())._handle, *args, stream)
    if type(r) is int:
        raise FAError(r, where)
    return r


def fa_fwd_span(q, k, v, key_begin, key_end, out, lse, softcap=0.0, slopes=None, scale=None,
                stream=None):
    """Call fa_fwd_span: row i of batch b sees keys key_begin[b, i] <= j < key_end[b, i]
    (int32 [B,Sq]); scores capped by softcap (0: not) and biased by
    -slopes[h] * |i + Skv - Sq - j| (float32 [Hq], or None)."""
    _given(out=out, lse=lse)
    _call("span_forward", "fa_fwd_span", q, k, v, key_begin, key_end, out, lse, softcap, slopes,
          scale, stream=stream)


def _given(**named):
    """The tensors a caller of the C-named functions has to bring."""
    for name, t in named.items():
        if t is None:
            raise ValueError(f"{name} must be a tensor")


def fa_bwd_span_workspace_bytes(B, Hq, Hkv, Sq, Skv, d) -> int:
    return int(lib().fa_bwd_span_workspace_bytes(B, Hq, Hkv, Sq, Skv, d))


def fa_bwd_span(q, k, v, key_begin, key_end, out, dout, lse, dq, dk, dv, workspace, softcap=0.0,
                slopes=None, scale=None, stream=None):
    """Call fa_bwd_span; `workspace` is a device tensor of at least
    fa_bwd_span_workspace_bytes(...) bytes."""
    _given(dq=dq, dk=dk, dv=dv, workspace=workspace)
    _call("span_backward", "fa_bwd_span", q, k, v, key_begin, key_end, out, dout, lse, dq, dk, dv,
          workspace, softcap, slopes, scale, stream=stream)


def attention_span_forward(q, k, v, key_begin, key_end, softcap=0.0, slopes=None, scale=None,
                           stream=None):
    """Allocate out and lse and run fa_fwd_span. Returns (out, lse)."""
    return _call("span_forward", "fa_fwd_span", q, k, v, key_begin, key_end, None, None, softcap,
                 slopes, scale, stream=stream)


def attention_span_backward(q, k, v, out, dout, lse, key_begin, key_end, softcap=0.0,
                            slopes=None, scale=None, workspace=None, stream=None):
    """Allocate dq, dk, dv (and a workspace unless given) and run fa_bwd_span."""
    return _call("span_backward", "fa_bwd_span", q, k, v, key_begin, key_end, out, dout, lse, None,
                 None, None, workspace, softcap, slopes, scale, stream=stream)


def key_spans(B, Sq, Skv=None, *, causal=True, window=0, doc_lens=None, prefix_lens=None,
              kv_lens=None, device=None):
    """(key_begin, key_end), int32 [B, Sq], of the usual masks, combined. Query row i stands at
    position i + Skv - Sq.

    causal       up to the row's own position
    window       only the last `window` keys up to the row's position (0: all)
    doc_lens     lengths of the documents packed along the keys, the same in every sequence
                 (a list or tensor) or one list per sequence: a row sees its own document only, and rows
                 outside all documents see nothing
    prefix_lens  one number, or one per sequence: the first keys (of the row's document, with
                 doc_lens) that every row sees although they lie after it
    kv_lens      one number, or one per sequence: real keys; rows and keys past them are padding
    """
    Skv = Sq if Skv is None else Skv
    if window < 0:
        raise ValueError("window must be >= 0")
    pos = torch.arange(Sq, dtype=torch.int64)[None, :].expand(B, Sq) + (Skv - Sq)

    def column(x):
        t = torch.as_tensor(x, dtype=torch.int64).reshape(-1)
        if t.numel() not in (1, B):
            raise ValueError(f"one value or {B} wanted, not {t.numel()}")
        if (t < 0).any():
            raise ValueError("lengths must be >= 0")
        return t[:, None].expand(B, 1)

    begin, last = torch.zeros(B, Sq, dtype=torch.int64), torch.full((B, Sq), Skv)
    if doc_lens is not None:
        rows = [x.tolist() if isinstance(x, torch.Tensor) else x for x in doc_lens]
        if not rows or not isinstance(rows[0], (list, tuple)):
            rows = [rows] * B
        if len(rows) != B:
            raise ValueError(f"one list of lengths or {B} wanted, not {len(rows)}")
        for b, lens in enumerate(rows):
            if any(n < 0 for n in lens) or sum(lens) > Skv:
                raise ValueError("documents must have lengths >= 0 and fit into the keys")
            ends = torch.tensor(list(lens), dtype=torch.int64).cumsum(0)
            which = torch.searchsorted(ends, pos[b].contiguous(), right=True)
            edges = torch.cat((torch.zeros(1, dtype=torch.int64), ends, ends[-1:] if lens else
                               torch.zeros(1, dtype=torch.int64)))
            begin[b], last[b] = edges[which], edges[which + 1]
        last = torch.where(pos < 0, begin, last)   # fewer keys than rows: before every document
    if kv_lens is not None:
        n = column(kv_lens)
        last = torch.where(pos < n, torch.minimum(last, n), torch.zeros_like(last))
    end = torch.minimum(last, pos + 1) if causal else last
    first = begin
    if window:
        begin = torch.maximum(begin, pos + 1 - int(window))
    if prefix_lens is not None:
        if window:
            raise ValueError("a prefix and a window together are not one range of keys")
        end = torch.maximum(end, torch.minimum(first + column(prefix_lens), last))
    empty = end <= begin
    begin, end = (torch.where(empty, torch.zeros_like(x), x).to(torch.int32).contiguous()
                  for x in (begin, end))
    return begin.to(device), end.to(device)


# ------------------------------------------------------ ragged paged cache --
def fa_fwd_ragged_paged_workspace_bytes(B, Hq, Hkv, Sq, d, block_size, max_blocks) -> int:
    return int(lib().fa_fwd_ragged_paged_workspace_bytes(B, Hq, Hkv, Sq, d, block_size, max_blocks))


def fa_fwd_ragged_paged(q, k_cache, v_cache, block_table, seq_lens, out, lse, workspace,
                        window=0, softcap=0.0, slopes=None, scale=None, stream=None):
    """Call fa_fwd_ragged_paged: q [B,Hq,Sq,d], the last Sq tokens of each sequence;
    k_cache/v_cache [num_blocks,Hkv,block_size,d]; block_table int32 [B,max_blocks];
    seq_lens int32 [B]; `workspace` a device tensor of at least
    fa_fwd_ragged_paged_workspace_bytes(...) bytes."""
    _given(out=out, lse=lse, workspace=workspace)
    _call("ragged", "fa_fwd_ragged_paged", q, k_cache, v_cache, block_table, seq_lens, out, lse,
          workspace, window, softcap, slopes, scale, stream=stream)


def decode_forward_ragged(q, k_cache, v_cache, block_table, seq_lens, window=0, softcap=0.0,
                          slopes=None, scale=None, stream=None):
    """Allocate out, lse and the workspace and run fa_fwd_ragged_paged. Returns (out, lse)."""
    return _call("ragged", "fa_fwd_ragged_paged", q, k_cache, v_cache, block_table, seq_lens, None,
                 None, None, window, softcap, slopes, scale, stream=stream)


# ------------------------------------------------ query / key preparation --
def rope_inv_freq(rope_dim, base=10000.0, scaling="none", factor=1.0, trained_len=8192,
                  low_turns=1.0, high_turns=32.0):
    """Rotary frequencies (float64 [rope_dim / 2], radians a position) and the rope_scale that
    goes with them, as (inv_freq, rope_scale). `scaling` stretches a trained context of
    trained_len positions by `factor`:

    none    base^(-2i / rope_dim)
    linear  all frequencies divided by factor (positions interpolated)
    base    the base raised so that the slowest frequency is divided by factor
    parts   YaRN as the paper writes it (Peng et al., 2023): frequencies that turn more than
            high_turns times within trained_len stay, those that turn less than low_turns times
            are divided by factor, in between linear in the number of turns;
            rope_scale = 0.1 ln(factor) + 1. (Programs that run published checkpoints often take
            a ramp linear in the pair's index instead, which gives other frequencies in between:
            pass such a table to rope_turns.)
    """
    if rope_dim < 2 or rope_dim % 2:
        raise ValueError("rope_dim must be even and positive")
    if not (factor >= 1.0 and base > 1.0 and high_turns > low_turns):
        raise ValueError("factor must be >= 1, base > 1 and high_turns > low_turns")
    if scaling == "base" and rope_dim > 2:
        base = base * factor ** (rope_dim / (rope_dim - 2))
    f = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)
    if scaling in ("none", "base"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        n = f * trained_len / (2 * math.pi)
        keep = ((n - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


def rope_turns(inv_freq, device=None):
    """The table the rotary calls take: int64 [rope_dim / 2], the frequencies (radians a
    position) as turns a position in units of 2^-64, modulo a turn."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").reshape(-1)
    out = []
    for x in f.tolist():
        if not math.isfinite(x):
            raise ValueError("frequencies must be finite")
        u = int(round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64)) % (1 << 64)
        out.append(u - (1 << 64) if u >= 1 << 63 else u)   # the same bits, signed
    return torch.tensor(out, dtype=torch.int64, device=device)


def fa_qk_norm_rope(q, k, q_out, k_out, turns, positions=None, q_weight=None, k_weight=None,
                    eps=1e-6, interleaved=False, rope_scale=1.0, stream=None):
    """Call fa_qk_norm_rope on views q, q_out [B,Hq,S,d] and k, k_out [B,Hkv,S,d] (any strides
    but the last); turns as from rope_turns (rope_dim = 2 * its length; None: no rotation);
    positions int32 [B,S] or None (row s at position s); both weights [d] or neither."""
    _given(q_out=q_out, k_out=k_out)
    _call("norm_rope", "fa_qk_norm_rope", q, k, q_out, k_out, turns, positions, q_weight, k_weight,
          eps, interleaved, rope_scale, stream=stream)


def fa_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hkv, S, d, norm=True) -> int:
    return int(lib().fa_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hkv, S, d, int(bool(norm))))


def fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, workspace, turns,
                        positions=None, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, rope_scale=1.0, stream=None):
    """Call fa_qk_norm_rope_bwd: views as for fa_qk_norm_rope; dq_weight, dk_weight float32 [d]
    and `workspace` (fa_qk_norm_rope_bwd_workspace_bytes bytes) with weights, else None."""
    _call("norm_rope_bwd", "fa_qk_norm_rope_bwd", dq_out, dk_out, q, k, dq, dk, dq_weight,
          dk_weight, workspace, turns, positions, q_weight, k_weight, eps, interleaved, rope_scale,
          False, stream=stream)


def fa_qk_norm_rope_append(q, k, v, q_out, k_cache, v_cache, block_table, seq_lens, turns,
                           q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                           rope_scale=1.0, stream=None):
    """Call fa_qk_norm_rope_append: the last Sq tokens of sequences of seq_lens tokens; views q,
    q_out [B,Hq,Sq,d], k, v [B,Hkv,Sq,d]; caches [num_blocks,Hkv,block_size,d] written in place."""
    _given(q_out=q_out)
    _call("append", "fa_qk_norm_rope_append", q, k, v, q_out, k_cache, v_cache, block_table,
          seq_lens, turns, q_weight, k_weight, eps, interleaved, rope_scale, stream=stream)


def qk_norm_rope_forward(q, k, turns, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, rope_scale=1.0, stream=None):
    """Allocate contiguous q_out [B,Hq,S,d] and k_out [B,Hkv,S,d] (as the attention calls take
    them) and run fa_qk_norm_rope. Returns (q_out, k_out)."""
    return _call("norm_rope", "fa_qk_norm_rope", q, k, None, None, turns, positions, q_weight,
                 k_weight, eps, interleaved, rope_scale, stream=stream)


def qk_norm_rope_backward(dq_out, dk_out, q, k, turns, positions=None, q_weight=None,
                          k_weight=None, eps=1e-6, interleaved=False, rope_scale=1.0, dq=None,
                          dk=None, stream=None):
    """Allocate dq, dk (unless given, e.g. as views of a packed gradient; else laid out
    [B, S, H, d] in memory, as projections give q and k) and, with weights, the float32 weight
    gradients, and run fa_qk_norm_rope_bwd. Returns (dq, dk, dq_weight, dk_weight), the last two
    None without weights. Without weights q and k are not read and may be None."""
    return _call("norm_rope_bwd", "fa_qk_norm_rope_bwd", dq_out, dk_out, q, k, dq, dk, None, None,
                 None, turns, positions, q_weight, k_weight, eps, interleaved, rope_scale,
                 True, stream=stream)


def qk_norm_rope_append(q, k, v, k_cache, v_cache, block_table, seq_lens, turns, q_weight=None,
                        k_weight=None, eps=1e-6, interleaved=False, rope_scale=1.0, stream=None):
    """Allocate q_out (contiguous [B,Hq,Sq,d]) and run fa_qk_norm_rope_append, which writes the
    tokens' keys and values into the caches. Returns q_out."""
    return _call("append", "fa_qk_norm_rope_append", q, k, v, None, k_cache, v_cache, block_table,
                 seq_lens, turns, q_weight, k_weight, eps, interleaved, rope_scale, stream=stream)


def decode_step_ragged(q, k, v, k_cache, v_cache, block_table, seq_lens, turns, q_weight=None,
                       k_weight=None, eps=1e-6, interleaved=False, rope_scale=1.0, window=0,
                       softcap=0.0, slopes=None, scale=None, stream=None):
    """One attention step of a serving loop: qk_norm_rope_append of the new tokens' projections
    q [B,Hq,Sq,d], k, v [B,Hkv,Sq,d], then decode_forward_ragged over the cache with them.
    seq_lens counts the new tokens. Returns (out, lse). Arguments that either refuses are refused
    before the caches are written."""
    return _call("step", "decode_step_ragged", q, k, v, k_cache, v_cache, block_table, seq_lens,
                 turns, q_weight, k_weight, eps, interleaved, rope_scale, window, softcap, slopes,
                 scale, stream=stream)


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024   # FA_NOALLOC_SCRATCH_BYTES in include/fa.h


def fa_bwd_noalloc(q, k, v, out, dout, lse, dq, dk, dv, causal=True, scale=None, stream=None):
    """Call fa_bwd_noalloc: fa_bwd without a workspace, for callers that cannot
    allocate device memory; the scratch is a fixed array inside libfa (see
    include/fa.h for its size, sharing and ordering rules)."""
    L = lib()
    fn = L.fa_bwd_noalloc
    if fn.argtypes is None:
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        fn.argtypes = [vp] * 9 + [i32, i32, i32, i32, i32, i32, ctypes.c_float, i32, vp]
        fn.restype = i32
    _check_contig(q, k, v, out, dout, lse, dq, dk, dv)
    B, Hq, Hkv, S, d = _dims(q, k)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    with _on_device(q):   # the scratch array used is the current device's
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                _ptr(dv), B, Hq, Hkv, S, d, int(bool(causal)), scale,
                DTYPE_CODES.get(q.dtype, -1), _stream(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_bwd_noalloc")
