"""Python binding of libsparse_transformer_attn.so (factorized sparse attention, B200).

Argument marshalling only: every step of the forward and backward pass runs
in the library's CUDA kernels. PyTorch supplies device memory and the current
stream. The names mirror the C ABI in include/sparse_transformer_attn.h.
There is no fallback: if the shared library is missing the import of any
entry point raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsparse_transformer_attn.so")

ST_OK, ST_ERR_INVALID, ST_ERR_UNSUPPORTED, ST_ERR_CUDA, ST_ERR_DEVICE_TIMEOUT, ST_ERR_WORKSPACE = range(6)
ST_STRIDED, ST_FIXED, ST_DENSE_CAUSAL = 0, 1, 2
ST_HEADS_SPLIT, ST_HEADS_MERGED = 0, 1
ST_F32, ST_BF16, ST_F16 = 0, 1, 2
KINDS = {"strided": ST_STRIDED, "fixed": ST_FIXED, "dense": ST_DENSE_CAUSAL}
MODES = {"split": ST_HEADS_SPLIT, "merged": ST_HEADS_MERGED}
VIEWS = {0: "natural", 1: "summary", 2: "class"}
RULES = {0: "causal", 1: "band", 2: "block", 3: "stride", 4: "stride_far", 5: "summary",
         6: "summary_earlier"}

# Every symbol the header declares, with its ctypes signature.
_i32, _i64, _u64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
SIGNATURES = {
    "st_pattern_layout": (ctypes.c_int, [_P, _P, _P]),
    "st_pattern_layout_host": (ctypes.c_int, [_P, _P]),
    "st_layout_destroy": (None, [_P]),
    "st_layout_counts": (ctypes.c_int, [_P, _P, _P]),
    "st_layout_segment_info": (ctypes.c_int, [_P, _i32, _i32, _P, _P, _P]),
    "st_layout_export": (ctypes.c_int, [_P, _i32, _i32, _i32, _P, _P, _P, _P, _P]),
    "st_layout_rows": (ctypes.c_int, [_P, _i32, _i32, _P, _P]),
    "st_layout_nnz": (ctypes.c_int, [_P, _i32, _P]),
    "st_sparse_attn_fwd": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32,
                                          ctypes.c_float, _P, _P, _P, _P, _P, _P]),
    "st_sparse_attn_bwd_workspace": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32,
                                                    _P]),
    "st_sparse_attn_bwd": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32,
                                          ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                          _P, ctypes.c_size_t, _P]),
    "st_sparse_attn_fwd_heads": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32, _i32,
                                                _i32, ctypes.c_float, _P, _P, _P, _P, _P, _P]),
    "st_sparse_attn_bwd_heads": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32, _i32,
                                                _i32, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P,
                                                _P, _P, _P, ctypes.c_size_t, _P]),
    "st_sparse_attn_bwd_noalloc": (ctypes.c_int, [_P, ctypes.c_int, _i32, _i32, _i32, _i32,
                                                  ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P,
                                                  _P, _P]),
    "st_packed_attn_fwd_workspace": (ctypes.c_int, [_P, ctypes.c_int, _P, _P]),
    "st_packed_attn_fwd": (ctypes.c_int, [_P, ctypes.c_int, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                                          _P, _P, ctypes.c_size_t, _P]),
    "st_packed_attn_bwd_workspace": (ctypes.c_int, [_P, ctypes.c_int, _P, _P]),
    "st_packed_attn_bwd": (ctypes.c_int, [_P, ctypes.c_int, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                                          _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "st_paged_attn_workspace": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _i32, _P]),
    "st_paged_attn": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _i32, ctypes.c_float, _P, _P, _P, _P,
                                     _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "st_cache_append": (ctypes.c_int, [ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "st_last_device_status": (ctypes.c_int, [_P]),
    "st_set_wait_limit": (ctypes.c_int, [_u64, _i32]),
    "st_layout_launches": (ctypes.c_int, [_P, ctypes.c_int, _P, _P]),
    "st_kernel_timing": (ctypes.c_int, [_i32]),
    "st_kernel_elapsed_ms": (ctypes.c_int, [_i32, _P]),
    "st_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "st_version": (ctypes.c_char_p, []),
}


class _Desc(ctypes.Structure):
    _fields_ = [("kind", _i32), ("head_mode", _i32), ("T", _i32), ("l", _i32), ("c", _i32)]


class _PackedDesc(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("total", _i32), ("H", _i32), ("Hkv", _i32), ("d", _i32),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("dq_stride", _i64), ("dk_stride", _i64), ("dv_stride", _i64)]


class _CacheDesc(ctypes.Structure):
    _fields_ = [("num_pages", _i32), ("page_size", _i32), ("max_pages", _i32),
                ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64)]


class StatusError(RuntimeError):
    def __init__(self, code, where):
        self.code = int(code)
        msg = status_string(code) if _lib is not None else str(code)
        super().__init__(f"{where}: status {code} ({msg})")


_lib = None


def lib():
    """The loaded shared library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m factorized_sparse_self_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(code) -> str:
    return lib().st_status_string(int(code)).decode()


def _check(code, where):
    if code != ST_OK:
        raise StatusError(code, where)


def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Layout:
    """Owner of one st_layout (host copy, and the device copy unless host_only)."""

    def __init__(self, kind, mode, T, l, c=1, host_only=False, stream=None):
        self.kind = KINDS[kind] if isinstance(kind, str) else int(kind)
        self.mode = MODES[mode] if isinstance(mode, str) else int(mode)
        self.T, self.l, self.c = int(T), int(l), int(c)
        d = _Desc(self.kind, self.mode, self.T, self.l, self.c)
        h = ctypes.c_void_p()
        if host_only:
            _check(lib().st_pattern_layout_host(ctypes.byref(d), ctypes.byref(h)),
                   "st_pattern_layout_host")
        else:
            _check(lib().st_pattern_layout(ctypes.byref(d), ctypes.byref(h), _stream_ptr(stream)),
                   "st_pattern_layout")
        self.handle = h
        self.host_only = host_only

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.st_layout_destroy(h)
            self.handle = None

    def counts(self):
        a, b = _i32(), _i32()
        _check(lib().st_layout_counts(self.handle, ctypes.byref(a), ctypes.byref(b)),
               "st_layout_counts")
        return a.value, b.value

    def segment_info(self, hc, seg):
        qv, kv, r = _i32(), _i32(), _i32()
        _check(lib().st_layout_segment_info(self.handle, hc, seg, ctypes.byref(qv),
                                            ctypes.byref(kv), ctypes.byref(r)),
               "st_layout_segment_info")
        return qv.value, kv.value, r.value

    def nnz(self, hc):
        n = _i64()
        _check(lib().st_layout_nnz(self.handle, hc, ctypes.byref(n)), "st_layout_nnz")
        return n.value

    def launches(self, dtype):
        """(forward, backward) kernel launches per call for this dtype code."""
        f, b = _i32(), _i32()
        _check(lib().st_layout_launches(self.handle, dtype, ctypes.byref(f), ctypes.byref(b)),
               "st_layout_launches")
        return f.value, b.value

    # row lists of st_layout_rows
    ROWS_Q_ACC, ROWS_K_ACC, ROWS_Q_ZERO, ROWS_K_ZERO = 0, 1, 2, 3

    def rows(self, hc, which):
        """Natural rows of head class hc in row list `which` (st_layout_rows)."""
        n = _i64(0)
        _check(lib().st_layout_rows(self.handle, hc, which, None, ctypes.byref(n)),
               "st_layout_rows")
        out = np.zeros(max(n.value, 1), dtype=np.int32)
        n2 = _i64(out.size)
        _check(lib().st_layout_rows(self.handle, hc, which, out.ctypes.data_as(_P),
                                    ctypes.byref(n2)), "st_layout_rows")
        return out[:n.value]

    def export(self, hc, seg, transpose=False):
        """(ptr, idx, flags, live) numpy arrays of one segment (seg = -1: natural tiling)."""
        sizes = (_i64 * 2)(0, 0)
        code = lib().st_layout_export(self.handle, hc, seg, int(transpose), None, None, None,
                                      None, sizes)
        _check(code, "st_layout_export")
        ptr = np.zeros(sizes[0], dtype=np.int32)
        idx = np.zeros(max(sizes[1], 1), dtype=np.int32)
        flags = np.zeros(max(sizes[1], 1), dtype=np.uint8)
        live = np.zeros(max(sizes[1], 1), dtype=np.int32)
        sizes2 = (_i64 * 2)(sizes[0], max(sizes[1], 1))
        _check(lib().st_layout_export(self.handle, hc, seg, int(transpose),
                                      ptr.ctypes.data_as(_P), idx.ctypes.data_as(_P),
                                      flags.ctypes.data_as(_P), live.ctypes.data_as(_P), sizes2),
               "st_layout_export")
        n = sizes[1]
        return ptr, idx[:n], flags[:n], live[:n]


def st_pattern_layout(kind, mode, T, l, c=1, stream=None) -> Layout:
    return Layout(kind, mode, T, l, c, host_only=False, stream=stream)


def st_pattern_layout_host(kind, mode, T, l, c=1) -> Layout:
    return Layout(kind, mode, T, l, c, host_only=True)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return ST_F32
    if t.dtype == torch.bfloat16:
        return ST_BF16
    if t.dtype == torch.float16:
        return ST_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t, name, like=None):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if like is not None and (t.dtype != like.dtype or t.shape != like.shape):
        raise ValueError(f"{name} must match q in dtype and shape")
    return ctypes.c_void_p(t.data_ptr())


def st_sparse_attn_fwd(layout: Layout, q, k, v, scale=None, o=None, lse=None, stream=None,
                       heads=None):
    """O [B,H,T,d] (dtype of q) and LSE [B,H,T] float32 for all heads, or for
    heads = (begin, count) only (st_sparse_attn_fwd_heads; other heads' rows
    of o and lse are left as they are)."""
    import torch
    B, H, T, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    args = [_need(x, n, q) for x, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"))]
    sc = float(scale) if scale else 0.0
    if heads is None:
        code = lib().st_sparse_attn_fwd(layout.handle, _dtype_code(q), B, H, T, d, sc, args[0],
                                        args[1], args[2], args[3], _need(lse, "lse"),
                                        _stream_ptr(stream))
        _check(code, "st_sparse_attn_fwd")
    else:
        code = lib().st_sparse_attn_fwd_heads(layout.handle, _dtype_code(q), B, H, heads[0],
                                              heads[1], T, d, sc, args[0], args[1], args[2],
                                              args[3], _need(lse, "lse"), _stream_ptr(stream))
        _check(code, "st_sparse_attn_fwd_heads")
    return o, lse


def st_sparse_attn_bwd_workspace(layout: Layout, dtype, B, H, T, d) -> int:
    n = ctypes.c_size_t()
    code = lib().st_sparse_attn_bwd_workspace(layout.handle, dtype, B, H, T, d, ctypes.byref(n))
    _check(code, "st_sparse_attn_bwd_workspace")
    return n.value


def st_sparse_attn_bwd(layout: Layout, q, k, v, o, lse, dout, scale=None, workspace=None,
                       dq=None, dk=None, dv=None, stream=None, heads=None):
    """dQ, dK, dV (dtype of q), with P recomputed from LSE; for heads =
    (begin, count) only when given (st_sparse_attn_bwd_heads)."""
    import torch
    B, H, T, d = q.shape
    if workspace is None:
        nb = st_sparse_attn_bwd_workspace(layout, _dtype_code(q), B, H, T, d)
        workspace = torch.empty(nb, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    ptrs = [_need(x, n, q) for x, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"),
                                        (dq, "dq"), (dk, "dk"), (dv, "dv"))]
    sc = float(scale) if scale else 0.0
    ws = ctypes.c_void_p(workspace.data_ptr())
    if heads is None:
        code = lib().st_sparse_attn_bwd(layout.handle, _dtype_code(q), B, H, T, d, sc, ptrs[0],
                                        ptrs[1], ptrs[2], ptrs[3], _need(lse, "lse"), ptrs[4],
                                        ptrs[5], ptrs[6], ptrs[7], ws, workspace.numel(),
                                        _stream_ptr(stream))
        _check(code, "st_sparse_attn_bwd")
    else:
        code = lib().st_sparse_attn_bwd_heads(layout.handle, _dtype_code(q), B, H, heads[0],
                                              heads[1], T, d, sc, ptrs[0], ptrs[1], ptrs[2],
                                              ptrs[3], _need(lse, "lse"), ptrs[4], ptrs[5],
                                              ptrs[6], ptrs[7], ws, workspace.numel(),
                                              _stream_ptr(stream))
        _check(code, "st_sparse_attn_bwd_heads")
    return dq, dk, dv


def st_sparse_attn_bwd_noalloc(layout: Layout, q, k, v, o, lse, dout, dq, dk, dv, scale=None,
                               stream=None):
    """Backward for callers that cannot allocate device memory: same result as
    st_sparse_attn_bwd, with the scratch in a fixed 64 MiB library-owned
    device array instead of a caller workspace. The caller passes every output
    buffer; nothing is allocated here or in the library. Calls whose GPU work
    overlaps share that array and race, so serialise them."""
    B, H, T, d = q.shape
    ptrs = [_need(x, n, q) for x, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"),
                                        (dq, "dq"), (dk, "dk"), (dv, "dv"))]
    code = lib().st_sparse_attn_bwd_noalloc(layout.handle, _dtype_code(q), B, H, T, d,
                                            float(scale) if scale else 0.0, ptrs[0], ptrs[1],
                                            ptrs[2], ptrs[3], _need(lse, "lse"), ptrs[4], ptrs[5],
                                            ptrs[6], ptrs[7], _stream_ptr(stream))
    _check(code, "st_sparse_attn_bwd_noalloc")
    return dq, dk, dv


# ---- ragged sequences, grouped heads, paged caches ----------------------------------------


class Pattern:
    """Kind, head mode, l and c of a pattern for sequences of any length (no layout is built)."""

    def __init__(self, kind, mode="merged", l=1, c=1):
        self.kind = KINDS[kind] if isinstance(kind, str) else int(kind)
        self.mode = MODES[mode] if isinstance(mode, str) else int(mode)
        self.l, self.c = int(l), int(c)

    def _desc(self, max_len):
        # a batch of empty sequences only has a longest one of 0
        return _Desc(self.kind, self.mode, int(max_len) or 1, self.l, self.c)


def st_pattern(kind, mode="merged", l=1, c=1) -> Pattern:
    """Pattern of the ragged and paged calls: "strided", "fixed" or "dense", "split" or "merged"
    heads, stride / block length l, summary count c (fixed)."""
    return Pattern(kind, mode, l, c)


def _tokens(t, name, q=None, heads=None):
    """Token stride of token rows [total, heads, d] (like q: its d, dtype, device and rows): the
    heads of a token lie d apart, tokens any multiple of d."""
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, heads, d]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if q is not None:
        if t.dtype != q.dtype or t.device != q.device:
            raise ValueError(f"{name} must match q in dtype and device")
        if d != q.shape[2] or n != q.shape[0] or (heads is not None and h != heads):
            raise ValueError(f"{name} has the wrong shape {tuple(t.shape)}")
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name} must have the heads of a token contiguous")
    if n <= 1:
        return h * d
    if s0 < h * d or s0 % d:
        raise ValueError(f"{name}: tokens must be a multiple of d = {d} elements apart")
    return s0


def _ints(t, name, n, like):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} values on {like.device}")
    return t.data_ptr()


def _rows_out(t, name, shape, dtype, like):
    if t.shape != shape or t.dtype != dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {like.device}")
    return t.data_ptr()


def _call_stream(stream, like):
    """The CUDA stream of a call (an integer)."""
    import torch
    dev = like.device.index
    if torch.cuda.current_device() != dev:
        raise ValueError(f"tensors are on {like.device}, which is not the current device")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _raw_stream(dev):
    # the current stream without the object around it (a fifth of the binding's time)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _on(stream):
    """What a call allocates for itself belongs to its stream: the memory is not handed out again
    before the call's work is done."""
    import torch
    return torch.cuda.stream(stream)


def _outputs(q, o, lse):
    import torch
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = q.new_empty(q.shape[:2], dtype=torch.float32)
    return o, lse


def _work(workspace, nbytes, like):
    """A workspace of nbytes, the caller's if given (None: none needed)."""
    import torch
    if workspace is None:
        return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the tensors' device")
    return workspace


def _work_args(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _packed_desc(q, k, v, cu_seqlens):
    qs = _tokens(q, "q")
    ks = _tokens(k, "k", q)
    total, H, d = q.shape
    Hkv = k.shape[1]
    return _PackedDesc(cu_seqlens.numel() - 1, total, H, Hkv, d, qs, ks, _tokens(v, "v", q, Hkv), 0,
                       0, 0)


def _packed_workspace(name, pat, code, x):
    n = ctypes.c_size_t()
    _check(getattr(lib(), name)(ctypes.byref(pat), code, ctypes.byref(x), ctypes.byref(n)), name)
    return n.value


def st_packed_attn_fwd_workspace(pattern: Pattern, q, k, v, cu_seqlens, max_len) -> int:
    return _packed_workspace("st_packed_attn_fwd_workspace", pattern._desc(max_len), _dtype_code(q),
                             _packed_desc(q, k, v, cu_seqlens))


def st_packed_attn_fwd(pattern: Pattern, q, k, v, cu_seqlens, max_len, scale=None, o=None, lse=None,
                       workspace=None, stream=None):
    """Attention over packed sequences of any lengths: q [total, H, d], k, v [total, Hkv, d] (head h
    reads key/value head h // (H // Hkv); slices of a fused QKV tensor are fine), cu_seqlens int32
    [n + 1] on the device. max_len is the longest sequence expected (it only steers how work is
    split). Returns o [total, H, d] and lse float32 [total, H] (natural log); token rows of no
    sequence are not written."""
    import torch
    x = _packed_desc(q, k, v, cu_seqlens)
    cu = _ints(cu_seqlens, "cu_seqlens", x.n_seqs + 1, q)
    code, pat = _dtype_code(q), pattern._desc(max_len)
    nb = _packed_workspace("st_packed_attn_fwd_workspace", pat, code, x)
    sp = _call_stream(stream, q)
    if stream is None:
        (o, lse), work = _outputs(q, o, lse), _work(workspace, nb, q)
    else:
        with _on(stream):
            (o, lse), work = _outputs(q, o, lse), _work(workspace, nb, q)
    _check(lib().st_packed_attn_fwd(ctypes.byref(pat), code, ctypes.byref(x),
                                    float(scale) if scale else 0.0, q.data_ptr(), k.data_ptr(),
                                    v.data_ptr(), cu, _rows_out(o, "o", q.shape, q.dtype, q),
                                    _rows_out(lse, "lse", q.shape[:2], torch.float32, q),
                                    *_work_args(work), sp), "st_packed_attn_fwd")
    return o, lse


def st_packed_attn_bwd_workspace(pattern: Pattern, q, k, v, cu_seqlens, max_len) -> int:
    return _packed_workspace("st_packed_attn_bwd_workspace", pattern._desc(max_len), _dtype_code(q),
                             _packed_desc(q, k, v, cu_seqlens))


def st_packed_attn_bwd(pattern: Pattern, q, k, v, o, lse, dout, cu_seqlens, max_len, scale=None,
                       workspace=None, dq=None, dk=None, dv=None, stream=None):
    """dq [total, H, d], dk, dv [total, Hkv, d] of st_packed_attn_fwd (dtype of q; given tensors may
    be slices of a fused gradient). Rows of no sequence are not written."""
    import torch
    x = _packed_desc(q, k, v, cu_seqlens)
    cu = _ints(cu_seqlens, "cu_seqlens", x.n_seqs + 1, q)
    code, pat = _dtype_code(q), pattern._desc(max_len)
    nb = _packed_workspace("st_packed_attn_bwd_workspace", pat, code, x)
    sp = _call_stream(stream, q)

    def buffers():
        like = [torch.empty_like(t, memory_format=torch.contiguous_format) if g is None else g
                for t, g in ((q, dq), (k, dk), (v, dv))]
        return like, _work(workspace, nb, q)

    if stream is None:
        (dq, dk, dv), work = buffers()
    else:
        with _on(stream):
            (dq, dk, dv), work = buffers()
    x.dq_stride = _tokens(dq, "dq", q, x.H)
    x.dk_stride = _tokens(dk, "dk", q, x.Hkv)
    x.dv_stride = _tokens(dv, "dv", q, x.Hkv)
    _check(lib().st_packed_attn_bwd(ctypes.byref(pat), code, ctypes.byref(x),
                                    float(scale) if scale else 0.0, q.data_ptr(), k.data_ptr(),
                                    v.data_ptr(), _rows_out(o, "o", q.shape, q.dtype, q),
                                    _rows_out(lse, "lse", q.shape[:2], torch.float32, q),
                                    _rows_out(dout, "dout", q.shape, q.dtype, q), cu,
                                    dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *_work_args(work),
                                    sp), "st_packed_attn_bwd")
    return dq, dk, dv


def _cache_desc(k_cache, v_cache, page_table, like):
    d = like.shape[2]
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dim() != 4 or t.shape[3] != d or t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{name} must be [pages, page_size, Hkv, {d}], of {like.dtype} on "
                             f"{like.device}")
    n, size, Hkv, _ = k_cache.shape
    s = k_cache.stride()
    if k_cache.shape != v_cache.shape or s != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if s[3] != 1 and d > 1:
        raise ValueError("the caches must be contiguous in their last dimension")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [sequences, pages]")
    return _CacheDesc(n, size, page_table.shape[1], s[0], s[1], s[2]), Hkv


def _paged_args(q, k_cache, v_cache, page_table, cu_q, kv_lens):
    qs = _tokens(q, "q")
    S = cu_q.numel() - 1
    c, Hkv = _cache_desc(k_cache, v_cache, page_table, q)
    x = _PackedDesc(S, q.shape[0], q.shape[1], Hkv, q.shape[2], qs, 0, 0, 0, 0, 0)
    return x, c, (_ints(page_table, "page_table", S * c.max_pages, q), _ints(cu_q, "cu_q", S + 1, q),
                  _ints(kv_lens, "kv_lens", S, q))


def _paged_workspace(pat, code, x, c, max_q):
    n = ctypes.c_size_t()
    _check(lib().st_paged_attn_workspace(ctypes.byref(pat), code, ctypes.byref(x), ctypes.byref(c),
                                         max_q, ctypes.byref(n)), "st_paged_attn_workspace")
    return n.value


def st_paged_attn_workspace(pattern: Pattern, q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q,
                            max_kv) -> int:
    x, c, _ = _paged_args(q, k_cache, v_cache, page_table, cu_q, kv_lens)
    return _paged_workspace(pattern._desc(max_kv), _dtype_code(q), x, c, int(max_q) or 1)


def st_paged_attn(pattern: Pattern, q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv,
                  scale=None, o=None, lse=None, workspace=None, stream=None):
    """Attention of the newest tokens q [total, H, d] of every sequence (rows cu_q[s] ..
    cu_q[s + 1] - 1; one each in a decoding step) over the cache [pages, page_size, Hkv, d] that
    holds their keys and values already (st_cache_append): page_table int32 [n, max_pages], kv_lens
    int32 [n], the new tokens included. max_q and max_kv, the most new tokens and keys of a sequence
    expected, only steer how work is split. Returns o [total, H, d], lse float32 [total, H]."""
    import torch
    x, c, (pt, cu, kv) = _paged_args(q, k_cache, v_cache, page_table, cu_q, kv_lens)
    code, pat, max_q = _dtype_code(q), pattern._desc(max_kv), int(max_q) or 1
    nb = _paged_workspace(pat, code, x, c, max_q)
    sp = _call_stream(stream, q)
    if stream is None:
        (o, lse), work = _outputs(q, o, lse), _work(workspace, nb, q)
    else:
        with _on(stream):
            (o, lse), work = _outputs(q, o, lse), _work(workspace, nb, q)
    _check(lib().st_paged_attn(ctypes.byref(pat), code, ctypes.byref(x), ctypes.byref(c), max_q,
                               float(scale) if scale else 0.0, q.data_ptr(), k_cache.data_ptr(),
                               v_cache.data_ptr(), pt, cu, kv,
                               _rows_out(o, "o", q.shape, q.dtype, q),
                               _rows_out(lse, "lse", q.shape[:2], torch.float32, q),
                               *_work_args(work), sp), "st_paged_attn")
    return o, lse


def st_cache_append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, stream=None):
    """Writes new keys and values k, v [total, Hkv, d] into the pages of the cache: new token t of n
    of sequence s goes to position kv_lens[s] - n + t (kv_lens counts the new tokens)."""
    ks = _tokens(k, "k")
    total, Hkv, d = k.shape
    vs = _tokens(v, "v", k, Hkv)
    S = cu_seqlens.numel() - 1
    c, cache_heads = _cache_desc(k_cache, v_cache, page_table, k)
    if cache_heads != Hkv:
        raise ValueError("k and the cache differ in their number of heads")
    x = _PackedDesc(S, total, Hkv, Hkv, d, 0, ks, vs, 0, 0, 0)
    sp = _call_stream(stream, k)
    _check(lib().st_cache_append(_dtype_code(k), ctypes.byref(x), ctypes.byref(c), k.data_ptr(),
                                 v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 _ints(page_table, "page_table", S * c.max_pages, k),
                                 _ints(cu_seqlens, "cu_seqlens", S + 1, k),
                                 _ints(kv_lens, "kv_lens", S, k), sp), "st_cache_append")


def st_last_device_status(stream=None) -> int:
    return int(lib().st_last_device_status(_stream_ptr(stream)))


def st_set_wait_limit(ns: int, force_timeout: bool = False) -> None:
    _check(lib().st_set_wait_limit(int(ns), int(bool(force_timeout))), "st_set_wait_limit")


def st_kernel_timing(enable: bool) -> None:
    _check(lib().st_kernel_timing(int(bool(enable))), "st_kernel_timing")


def st_kernel_elapsed_ms(kernel: int) -> float:
    ms = ctypes.c_float()
    _check(lib().st_kernel_elapsed_ms(int(kernel), ctypes.byref(ms)), "st_kernel_elapsed_ms")
    return ms.value


def st_version() -> str:
    return lib().st_version().decode()
