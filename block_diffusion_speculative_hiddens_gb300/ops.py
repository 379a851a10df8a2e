"""Operators of a caller's own target model: rotary positions, the append to a
paged cache, and the attention of new tokens over it.

The library drafts and accepts; verifying is the caller's target, of any depth
and in the caller's own engine.  In every layer of it these calls go from the
projections' q, k and v (or, in a layer that normalises each head of q and k,
from what that norm gives) to the attention's output:

    plan = RopePlan(128, 1e6)                              # once a model
    cache = PagedCache(k_pool, v_pool, page_table)         # once a layer
    q = append(cache, k, v, cu_rows, ctx_len, plan=plan, q=q)
    o = attention(cache, q, cu_rows, ctx_len)

for a ragged batch of single tokens, verify blocks and prompt chunks: rows
cu_rows[b] .. cu_rows[b+1]-1 are sequence b's, at positions ctx_len[b] and on.
The C entry points, their argument structs, limits and device-side checks are
in include/dflash.h; this module checks the tensors (ValueError) and passes
their pointers and strides.  Calls go to the current stream of the tensors'
device (or `stream`), enqueue and return, and may be captured into a graph;
outputs that are not given are allocated on that stream.  With `stream`, the
tensors are ready on it and stay allocated until it is done, as for any work on
a stream of one's own.  Outputs that are given may be their own input (in
place); over anything else of the call, or over themselves, they are refused
(ValueError, or DflashError from the C entry).  The calls record nothing for
autograd: tensors that require a gradient are refused while gradients are
recorded.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from .binding import DflashError, load

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_KINDS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "llama3": 4, "factors": 5}
MAX_PAIRS = 128


class RopeConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rotary_dim", "interleaved", "scaling", "original_len")] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "beta_fast", "beta_slow", "low_freq", "high_freq",
                                       "attention_factor")] + [("factors", ctypes.POINTER(ctypes.c_double))]


class _Plan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turn", ctypes.c_uint64 * MAX_PAIRS)]


# The argument structs of include/dflash.h, packed with native alignment.
_ROWS = "Pqq"
_ROPE = struct.Struct("@" + 4 * _ROWS + "P7i0q")
_CACHE = struct.Struct("@PP6qPqP7i0q")
_APPEND = struct.Struct("@" + 4 * _ROWS + "PP4i0q")
_ATTENTION = struct.Struct("@" + 2 * _ROWS + "PqqPPPPq5if0q")
_NONE = (0, 0, 0)


def _int32(v, what):
    if v != int(v) or not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{what}: expected a 32-bit whole number, got {v}")
    return int(v)


class RopePlan:
    """The rotation of a model's heads: `rotary_dim` leading dims in pairs
    (i, i + rotary_dim/2), or (2i, 2i+1) if interleaved, at angle
    position * theta^(-2i/rotary_dim), scaled for long contexts by `scaling`:

        {"kind": "linear", "factor": s}
        {"kind": "ntk", "factor": s}
        {"kind": "yarn", "factor": s, "original_len": n, "beta_fast": 32, "beta_slow": 1[, "attention_factor": a]}
        {"kind": "llama3", "factor": s, "original_len": n, "low_freq_factor": 1, "high_freq_factor": 4}
        {"kind": "factors", "factors": [one a pair][, "attention_factor": a]}

    Held on the host; calls pass it to their kernels by value."""

    def __init__(self, rotary_dim: int, theta: float = 1e4, *, interleaved: bool = False, scaling: dict = None):
        rotary_dim = _int32(rotary_dim, "rotary_dim")
        s = dict(scaling or {"kind": "none"})
        kind = s.pop("kind", None)
        if kind not in _KINDS:
            raise ValueError(f"scaling: unknown kind {kind!r}; known: {sorted(_KINDS)}")
        known = {"none": (), "linear": ("factor",), "ntk": ("factor",),
                 "yarn": ("factor", "original_len", "beta_fast", "beta_slow", "attention_factor"),
                 "llama3": ("factor", "original_len", "low_freq_factor", "high_freq_factor"),
                 "factors": ("factors", "attention_factor")}[kind]
        if extra := sorted(set(s) - set(known)):
            raise ValueError(f"scaling: {kind} takes {list(known)}, got {extra}")
        need = {"factor", "original_len", "factors"} & set(known)
        if missing := sorted(need - set(s)):
            raise ValueError(f"scaling: {kind} needs {missing}")
        factors = None
        if kind == "factors":
            if len(s["factors"]) != rotary_dim // 2:
                raise ValueError(f"scaling: {len(s['factors'])} factors for {rotary_dim // 2} pairs")
            factors = (ctypes.c_double * len(s["factors"]))(*s["factors"])
        cfg = RopeConfig(rotary_dim=rotary_dim, interleaved=int(bool(interleaved)), scaling=_KINDS[kind],
                         original_len=_int32(s.get("original_len", 0), "original_len"), theta=theta,
                         factor=s.get("factor", 1.0),
                         beta_fast=s.get("beta_fast", 32.0), beta_slow=s.get("beta_slow", 1.0),
                         low_freq=s.get("low_freq_factor", 1.0), high_freq=s.get("high_freq_factor", 4.0),
                         attention_factor=s.get("attention_factor", 0.0),
                         factors=ctypes.cast(factors, ctypes.POINTER(ctypes.c_double)) if factors else None)
        self._c = _Plan()
        code = load().dflash_rope_init(ctypes.byref(cfg), ctypes.byref(self._c))
        if code:
            raise DflashError("dflash_rope_init", code)
        self._ref = ctypes.byref(self._c)
        self.rotary_dim = rotary_dim
        self.interleaved = bool(interleaved)
        self.amplitude = self._c.amplitude


def _graded(t):
    return getattr(t, "requires_grad", False)


def _no_gradient(what):
    """Autograd records nothing of a call: it is refused rather than cut out of a graph that is being recorded."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what}: requires a gradient, which this call does not record; use torch.no_grad()")


def _rows(t, what, dtype, device, rows=None, heads=None, dim=None):
    """A [rows, heads, head_dim] tensor's (pointer, row stride, head stride)."""
    if _graded(t):
        _no_gradient(what)
    shape, stride = t.shape, t.stride()
    if t.dtype is dtype and t.get_device() == device and len(shape) == 3 and stride[2] == 1 and \
            (rows is None or shape[0] == rows) and (heads is None or shape[1] == heads) and \
            (dim is None or shape[2] == dim):
        return t.data_ptr(), stride[0], stride[1]
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what}: expected {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    if len(shape) == 3 and stride[2] != 1:
        raise ValueError(f"{what}: the head dimension has stride {stride[2]}, expected 1")
    raise ValueError(f"{what}: expected [{'rows' if rows is None else rows}, {'heads' if heads is None else heads}, "
                     f"{'head_dim' if dim is None else dim}], got {list(shape)}")


def _i32(t, what, n, device):
    if t.dtype is not torch.int32 or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous int32 values on cuda:{device}, got {list(t.shape)} "
                         f"{t.dtype} on {t.device}")
    return t.data_ptr()


def _meet(x, y):
    """Whether two 16-bit views share an element; views of one buffer may
    interleave without meeting: heads of the same rows."""
    a, b = x.data_ptr(), y.data_ptr()
    ea = a + 2 * (1 + sum((n - 1) * s for n, s in zip(x.shape, x.stride())))
    eb = b + 2 * (1 + sum((n - 1) * s for n, s in zip(y.shape, y.stride())))
    return a < eb and b < ea and not _disjoint_heads(x, y)


def _no_overlap(out, src, what):
    """An output is its input itself, or apart from it; its heads of all rows lie apart from one another."""
    near, far = sorted((s, n) for s, n in zip(out.stride()[:2], out.shape[:2]))
    if near[1] > 1 and near[0] < out.shape[2] or \
            far[1] > 1 and far[0] < out.shape[2] + (near[1] - 1) * near[0]:
        raise ValueError(f"{what}: rows and heads overlap one another, strides {list(out.stride())}")
    if (out.data_ptr() != src.data_ptr() or out.stride() != src.stride()) and _meet(out, src):
        raise ValueError(f"{what}: overlaps its input without being it")


def _apart(out, other, what, name):
    """An output that the caller gave lies apart from what else the call reads or writes."""
    if _meet(out, other):
        raise ValueError(f"{what}: overlaps {name}")


def _disjoint_heads(x, y):
    """Whether two views with the same row stride hold different parts of every row."""
    row = x.stride(0)
    if row != y.stride(0) or row <= 0 or min(x.stride(1), y.stride(1)) < 0:
        return False
    wx, wy = ((t.shape[1] - 1) * t.stride(1) + t.shape[2] for t in (x, y))
    gap = (y.data_ptr() - x.data_ptr()) // 2 % row
    return wx <= gap and gap + wy <= row


# The current stream's handle; torch.cuda.current_stream builds an object for
# it, a microsecond of a call that takes ten.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(stream, device):
    if stream is None:
        return _current_stream(device)
    if stream.device.index != device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """Memory on the call's stream: the allocator hands it out again in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(out, src, rows, heads, dim, what, dtype, device, stream):
    """A call's output beside its input `src` -- the caller's, checked, or a new one -- and its pointer and strides."""
    if out is None:
        out = _empty((rows, heads, dim), dtype, src, stream)
        return out, (out.data_ptr(), heads * dim, dim)
    at = _rows(out, what, dtype, device, rows, heads, dim)
    _no_overlap(out, src, what)
    return out, at


def _cuda_half(t, what):
    device = t.get_device()
    if t.dtype not in _DTYPES or device < 0:
        raise ValueError(f"{what}: expected a float16 or bfloat16 CUDA tensor, got {t.dtype} on {t.device}")
    return device


def rope(plan: RopePlan, q, k, positions, *, backward: bool = False, q_out=None, k_out=None, stream=None):
    """Rotate q [rows, q_heads, head_dim] and k [rows, k_heads, head_dim] (or None)
    at positions [rows] int32; returns (q_out, k_out), new contiguous tensors
    unless given (an input itself: in place).  Any strides of rows and heads.
    backward=True applies the transposed rotation: the inputs' gradient from
    the outputs', for a caller's own autograd function."""
    device, dtype = _cuda_half(q, "q"), q.dtype
    raw = _raw_stream(stream, device)
    qs = _rows(q, "q", dtype, device)
    rows, hq, dim = q.shape
    given_q, given_k = q_out is not None, k_out is not None
    q_out, qo = _out(q_out, q, rows, hq, dim, "q_out", dtype, device, stream)
    ks, ko, hk = _NONE, _NONE, 0
    if k is not None:
        ks = _rows(k, "k", dtype, device, rows, None, dim)
        hk = k.shape[1]
        k_out, ko = _out(k_out, k, rows, hk, dim, "k_out", dtype, device, stream)
        if given_q:
            _apart(q_out, k, "q_out", "k")
        if given_k:
            _apart(k_out, q, "k_out", "q")
            if given_q:
                _apart(q_out, k_out, "q_out", "k_out")
    elif given_k:
        raise ValueError("k_out: given without k")
    args = _ROPE.pack(*qs, *ks, *qo, *ko, _i32(positions, "positions", rows, device), rows, hq, hk, dim, _DTYPES[dtype],
                      bool(backward), device)
    code = load().dflash_rope(plan._ref, args, raw)
    if code:
        raise DflashError("dflash_rope", code)
    return q_out, k_out


def _clear_word(device):
    """A zero that calls on any stream find, not only those behind the current one.
    A captured one is the graph's: each replay clears it, ahead of the graph's calls."""
    with torch.cuda.device(device):
        word = torch.zeros(1, dtype=torch.int32, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return word


class PagedCache:
    """Pools of K and V pages [n_pages, page_size, kv_heads, head_dim] (any
    order in memory: pass a permuted view) and a page table [batch, max_pages]
    int32 whose entry [b, p // page_size] is the page of sequence b's position
    p.  All of them are the caller's; the table's values may change between
    calls.  `status` collects the device-side checks of the calls on it: keep
    the cache as long as calls or captured graphs use it."""

    _graded = None  # a pool that requires a gradient

    def __init__(self, k_pool, v_pool, page_table):
        device = _cuda_half(k_pool, "k_pool")
        for what, t in (("k_pool", k_pool), ("v_pool", v_pool)):
            if t.dim() != 4 or t.shape != k_pool.shape or t.dtype is not k_pool.dtype or t.get_device() != device:
                raise ValueError(f"{what}: expected two pools [pages, page_size, kv_heads, head_dim] of one type on "
                                 f"one device, got {list(t.shape)} {t.dtype} on {t.device}")
            if t.stride(3) != 1:
                raise ValueError(f"{what}: the head dimension has stride {t.stride(3)}, expected 1")
        if page_table.dim() != 2 or page_table.dtype is not torch.int32 or page_table.get_device() != device or \
                page_table.stride(1) != 1:
            raise ValueError(f"page_table: expected int32 [batch, max_pages] with contiguous rows on cuda:{device}, "
                             f"got {list(page_table.shape)} {page_table.dtype} on {page_table.device}")
        table_stride, width = page_table.stride(0), page_table.shape[1]
        if table_stride < width:
            if page_table.shape[0] > 1:
                raise ValueError(f"page_table: rows overlap, stride {table_stride} for {width} entries; "
                                 "expanded tables: make them contiguous")
            table_stride = width  # of a single row
        self.k_pool, self.v_pool, self.page_table = k_pool, v_pool, page_table
        self._graded = "k_pool" if _graded(k_pool) else "v_pool" if _graded(v_pool) else None
        self.status = _clear_word(k_pool.device)
        self.device, self.dtype = device, k_pool.dtype
        self.n_pages, self.page_size, self.kv_heads, self.head_dim = k_pool.shape
        self.batch = page_table.shape[0]
        self._c = _CACHE.pack(
            k_pool.data_ptr(), v_pool.data_ptr(), *k_pool.stride()[:3], *v_pool.stride()[:3], page_table.data_ptr(),
            table_stride, self.status.data_ptr(), width, self.n_pages, self.page_size, self.kv_heads, self.head_dim,
            _DTYPES[self.dtype], device)

    def read_status(self) -> int:
        """DEV_* bits since the last call, and clears them.  Waits for the device:
        calls on every stream are in.  Not during a capture."""
        v = ctypes.c_uint32()
        code = load().dflash_paged_read_status(self._c, ctypes.byref(v))
        if code:
            raise DflashError("dflash_paged_read_status", code)
        return v.value


def _batch(cache, cu_rows, ctx_len):
    b = ctx_len.shape[0]
    if b > cache.batch:
        raise ValueError(f"ctx_len: {b} sequences, the page table has {cache.batch}")
    return b, _i32(cu_rows, "cu_rows", b + 1, cache.device), _i32(ctx_len, "ctx_len", b, cache.device)


def append(cache: PagedCache, k, v, cu_rows, ctx_len, *, plan: RopePlan = None, q=None, q_out=None, stream=None):
    """Write k and v [rows, kv_heads, head_dim] of a ragged batch into the cache
    at positions ctx_len[b] and on, k rotated by `plan` (None: as it is).  q
    [rows, q_heads, head_dim], if given, is rotated alike; returns q_out (None
    without q, which takes no q_out)."""
    device, dtype, dim = cache.device, cache.dtype, cache.head_dim
    if cache._graded:
        _no_gradient(cache._graded)
    raw = _raw_stream(stream, device)
    ks = _rows(k, "k", dtype, device, None, cache.kv_heads, dim)
    rows = k.shape[0]
    vs = _rows(v, "v", dtype, device, rows, cache.kv_heads, dim)
    b, cu, ctx = _batch(cache, cu_rows, ctx_len)
    qs, qo, hq = _NONE, _NONE, 0
    if q is not None:
        qs = _rows(q, "q", dtype, device, rows, None, dim)
        hq = q.shape[1]
        given = q_out is not None
        q_out, qo = _out(q_out, q, rows, hq, dim, "q_out", dtype, device, stream)
        if given:
            _apart(q_out, k, "q_out", "k")
            _apart(q_out, v, "q_out", "v")
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    args = _APPEND.pack(*ks, *vs, *qs, *qo, cu, ctx, rows, b, hq, 0)
    code = load().dflash_paged_append(cache._c, None if plan is None else plan._ref, args, raw)
    if code:
        raise DflashError("dflash_paged_append", code)
    return q_out


def attention(cache: PagedCache, q, cu_rows, ctx_len, *, kv_len=None, causal: bool = True, window: int = 0,
              scale: float = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [rows, q_heads, head_dim] over the cache: row i of sequence
    b, at position p = ctx_len[b] + i, sees the cached positions below kv_len[b]
    (None: ctx_len[b] + its rows, appended before), those up to p if causal,
    those above p - window if window > 0.  scale: 1/sqrt(head_dim) by default.
    out: q itself, or apart from it.  lse: float32 [rows, q_heads] output for the rows' log-sum-exp.  workspace:
    uint8, attention_workspace() bytes (0 for small calls); by default allocated
    for the call."""
    device, dtype, dim = cache.device, cache.dtype, cache.head_dim
    if cache._graded:
        _no_gradient(cache._graded)
    raw = _raw_stream(stream, device)
    qs = _rows(q, "q", dtype, device, None, None, dim)
    rows, hq, _ = q.shape
    b, cu, ctx = _batch(cache, cu_rows, ctx_len)
    kv = 0 if kv_len is None else _i32(kv_len, "kv_len", b, device)
    if out is None:
        out = _empty((rows, hq, dim), dtype, q, stream)
        os_ = out.data_ptr(), hq * dim, dim
    else:
        os_ = _rows(out, "out", dtype, device, rows, hq, dim)
        _no_overlap(out, q, "out")
    ls = _NONE
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.get_device() != device or tuple(lse.shape) != (rows, hq):
            raise ValueError(f"lse: expected float32 [{rows}, {hq}] on cuda:{device}, got {list(lse.shape)} {lse.dtype} "
                             f"on {lse.device}")
        if _graded(lse):
            _no_gradient("lse")
        ls = (lse.data_ptr(), lse.stride(0), lse.stride(1))
    lib = load()
    if workspace is None:
        nbytes = lib.dflash_paged_attention_workspace(cache._c, rows, b, hq)
        if nbytes:
            workspace = _empty(nbytes, torch.uint8, q, stream)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous uint8 on cuda:{device}, got {workspace.dtype} on "
                         f"{workspace.device}")
    else:
        nbytes = workspace.numel()
    args = _ATTENTION.pack(*qs, *os_, *ls, cu, ctx, kv, 0 if workspace is None else workspace.data_ptr(), nbytes,
                           rows, b, hq, bool(causal), window, dim ** -0.5 if scale is None else scale)
    code = lib.dflash_paged_attention(cache._c, args, raw)
    if code:
        raise DflashError("dflash_paged_attention", code)
    return out


def attention_workspace(cache: PagedCache, rows: int, batch: int, q_heads: int) -> int:
    """Bytes of workspace that attention() of this shape needs."""
    return load().dflash_paged_attention_workspace(cache._c, rows, batch, q_heads)
