"""Rotary positions, the 8-bit key/value cache and the attention over it.

The layer between a model's projections (gemv / gemm, which leave q, k, v in
fp32) and its output projection (which takes bf16):

    rope = mq.Rope(*mq.rope_frequencies(128, base=1e6))
    cache = mq.KVCache.allocate(pages=4096, heads=8, block=64, dim=128, fmt="int8")
    batch = mq.KVBatch(q_start, kv_len, page_table, rows=T, max_new=1)
    q_rot = mq.cache_append(cache, batch, k, v, q=q, rope=rope)
    out = mq.cache_attend(cache, batch, q_rot)

Like the rest of the package this is argument checking and marshalling; the
work runs in libmq.so.  Each call exists as a function and as a plan (RopePlan,
CacheAppendPlan, CacheAttendPlan), which checks and marshals once and then
makes one C call each time it is called, for loops bound by the launch rate.
A plan uses the tensors it was made of at their addresses and keeps them alive.
Calls must be made with the tensors' device as the current device.
"""

from __future__ import annotations

import ctypes
import math

from . import MQ_OK, MQError, _check, _need, _ptr, _same_device, _stream, lib

KV_FORMATS = {"int8": 0, "e4m3": 1}
_BF16, _F32 = 0, 1


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("block", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("table_pages", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


class _RopeSpec(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("factor", ctypes.c_double), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _StackAttention(ctypes.Structure):
    _fields_ = [("caches", ctypes.POINTER(_Cache)), ("batch", ctypes.POINTER(_Batch)),
                ("rope", ctypes.POINTER(_RopeSpec)), ("windows", ctypes.POINTER(ctypes.c_int64)),
                ("q_heads", ctypes.c_int64), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float)]


def declare(L):
    """Signatures of this module's entry points (called by lib())."""
    i64, vp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    C, B, R = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch), ctypes.POINTER(_RopeSpec)
    f32 = ctypes.c_float
    L.mq_rope.restype = i32
    L.mq_rope.argtypes = [R, vp, vp, i32, i64, i64, i64, i64, vp, i64, vp]
    L.mq_cache_append.restype = i32
    L.mq_cache_append.argtypes = [C, B, R, vp, vp, i64, vp, i64, i64, i32, vp, vp]
    L.mq_cache_read.restype = i32
    L.mq_cache_read.argtypes = [C, B, vp, vp, i32, vp]
    L.mq_cache_attend_workspace_bytes.restype = sz
    L.mq_cache_attend_workspace_bytes.argtypes = [C, B, i64, i64]
    L.mq_cache_attend.restype = i32
    L.mq_cache_attend.argtypes = [C, B, vp, i64, i64, f32, f32, i64, i32, vp, vp, vp, sz, vp]
    A = ctypes.POINTER(_StackAttention)
    L.mq_mixnmatch_attend_workspace_bytes.restype = sz
    L.mq_mixnmatch_attend_workspace_bytes.argtypes = [vp, i32, A, i64]
    L.mq_mixnmatch_attend.restype = i32
    L.mq_mixnmatch_attend.argtypes = [vp, i32, A, vp, i64, vp, vp, sz, vp]


# ---------------------------------------------------------------- argument checks

def _on_current(t, stream):
    """Work is launched on the current device: the tensors have to be there,
    and a stream given has to be one of it."""
    import torch

    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"mq: tensors on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"mq: a stream of {stream.device} for tensors on {t.device}")


def _empty(shape, dtype, device, stream):
    """A tensor that the call writes, from the memory of the stream it runs on
    (so that its memory is reused in that stream's order)."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows_view(x, name, heads=None, dim=None, rows=None):
    """x [rows, heads, dim] whose rows are contiguous and evenly spaced (it may
    be a part of wider rows): (type, row stride in entries)."""
    import torch

    _need(x, name, (torch.bfloat16, torch.float32))
    if x.dim() != 3:
        raise ValueError(f"mq: {name} must be [rows, heads, dim]")
    if not x.is_cuda:
        raise ValueError("mq: tensors must be on the GPU")
    t, h, d = x.shape
    for got, want, what in ((t, rows, "rows"), (h, heads, "heads"), (d, dim, "dim")):
        if want is not None and got != want:
            raise ValueError(f"mq: {name} has {got} {what}, expected {want}")
    if (d > 1 and x.stride(2) != 1) or (h > 1 and x.stride(1) != d):
        raise ValueError(f"mq: the rows of {name} must be contiguous")
    stride = x.stride(0) if t > 1 else h * d
    if stride < h * d:
        raise ValueError(f"mq: the rows of {name} overlap")
    return (_F32 if x.dtype == torch.float32 else _BF16), stride


def _addr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------- what a user keeps

def rope_frequencies(rot: int, base: float = 10000.0, scaling=None, device="cuda"):
    """(freq float64 [rot / 2] on `device`, factor) for Rope: base^(-2i/rot)
    radians a position, and the scaling of a context longer than the trained one:

      None                                          as they are, factor 1
      {"kind": "linear", "factor": f}               every frequency / f
      {"kind": "base", "factor": f}                 base * f^(rot / (rot - 2))
      {"kind": "bands", "factor": f, "trained": L, "low": 1, "high": 4}
            a pair that makes t = L freq / (2 pi) turns over the trained length
            keeps freq if t >= high, gets freq / f if t <= low, and a mix,
            linear in t, between
      {"kind": "yarn", "factor": f, "trained": L, "low": 1, "high": 32}
            the same, with the rotated entries multiplied by 0.1 ln f + 1
    """
    import torch

    if rot < 8 or rot % 8:
        raise ValueError("mq: rot must be a positive multiple of 8")
    if not base > 0:
        raise ValueError("mq: base must be positive")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    factor = 1.0
    if scaling is None:
        freq = base ** (-i / rot)
    else:
        kind, f = scaling.get("kind"), float(scaling.get("factor", 0.0))
        if not f > 0:
            raise ValueError("mq: scaling needs a positive factor")
        if kind == "linear":
            freq = base ** (-i / rot) / f
        elif kind == "base":
            freq = (base * f ** (rot / (rot - 2))) ** (-i / rot)
        elif kind in ("bands", "yarn"):
            freq = base ** (-i / rot)
            low = float(scaling.get("low", 1.0))
            high = float(scaling.get("high", 4.0 if kind == "bands" else 32.0))
            trained = float(scaling.get("trained", 0))
            if not (trained > 0 and high > low):
                raise ValueError("mq: scaling needs trained > 0 and high > low")
            keep = ((trained * freq / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
            freq = freq * (keep + (1 - keep) / f)
            if kind == "yarn":
                factor = 0.1 * math.log(f) + 1.0
        else:
            raise ValueError(f"mq: unknown scaling {kind!r}")
    return freq.to(device), factor


class Rope:
    """Rotary positions of a model: the frequencies of its rot / 2 pairs
    (float64, on the GPU), the pairs' layout (halves of the rotated part, or
    interleaved neighbours) and the factor of the rotated entries."""

    def __init__(self, freq, factor: float = 1.0, interleaved: bool = False):
        import torch

        _need(freq, "freq", (torch.float64,))
        if freq.dim() != 1:
            raise ValueError("mq: freq must be [rot / 2]")
        self.freq, self.factor, self.interleaved = freq, float(factor), bool(interleaved)
        self.rot = 2 * freq.numel()
        self.spec = _RopeSpec(_ptr(freq), self.factor, self.rot, int(self.interleaved))


class KVCache:
    """A paged 8-bit cache of one layer: k uint8 [pages, heads, block, dim],
    v uint8 [pages, heads, dim, block] (dim-major), k_scale and v_scale fp32
    [pages, heads]; value = code * scale; fmt "int8" or "e4m3"."""

    def __init__(self, k, v, k_scale, v_scale, fmt: str):
        import torch

        if fmt not in KV_FORMATS:
            raise ValueError(f"mq: unknown cache format {fmt!r}")
        _need(k, "k", (torch.uint8,))
        if k.dim() != 4:
            raise ValueError("mq: k must be [pages, heads, block, dim]")
        p, h, b, d = k.shape
        _need(v, "v", (torch.uint8,), shape=(p, h, d, b))
        _need(k_scale, "k_scale", (torch.float32,), shape=(p, h))
        _need(v_scale, "v_scale", (torch.float32,), shape=(p, h))
        _same_device(k, v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale, self.fmt = k, v, k_scale, v_scale, fmt
        self.pages, self.heads, self.block, self.dim = p, h, b, d
        self.c = _Cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), p, h, b, d,
                        KV_FORMATS[fmt])

    @classmethod
    def allocate(cls, pages: int, heads: int, block: int, dim: int, fmt: str = "int8",
                 device="cuda"):
        """An empty cache (all zeros)."""
        import torch

        z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device)  # noqa: E731
        f = lambda: torch.zeros((pages, heads), dtype=torch.float32, device=device)  # noqa: E731
        return cls(z(pages, heads, block, dim), z(pages, heads, dim, block), f(), f(), fmt)


class KVBatch:
    """The tokens of a call: sequence s owns rows q_start[s] .. q_start[s+1] - 1,
    its last tokens; kv_len[s] tokens of it are cached (these among them);
    page_table [seqs, pages of the longest].  All int32 on the GPU, read when
    the work runs.  rows: rows of q, k, v and the outputs; max_new: an upper
    bound of one sequence's rows."""

    def __init__(self, q_start, kv_len, page_table, rows: int, max_new: int):
        import torch

        i32 = (torch.int32,)
        _need(page_table, "page_table", i32)
        if page_table.dim() != 2:
            raise ValueError("mq: page_table must be [seqs, pages]")
        s, wide = page_table.shape
        _need(q_start, "q_start", i32, shape=(s + 1,))
        _need(kv_len, "kv_len", i32, shape=(s,))
        _same_device(q_start, kv_len, page_table)
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.rows, self.max_new, self.seqs = int(rows), int(max_new), s
        if not (0 <= self.rows < 1 << 31 and 1 <= self.max_new < 1 << 31):
            raise ValueError("mq: rows or max_new out of range")
        self.c = _Batch(_ptr(q_start), _ptr(kv_len), _ptr(page_table), self.rows, s, wide,
                        self.max_new)


class _Plan:
    """A checked and marshalled call: fn(*args), then `result`."""

    def _set(self, fn, name, args, result, keep, rows):
        self.fn, self.name, self.args, self.result = fn, name, args, result
        self.keep, self.rows = keep, rows

    def __call__(self):
        if self.rows:
            st = self.fn(*self.args)
            if st != MQ_OK:
                raise MQError(st, self.name)
        return self.result


# ---------------------------------------------------------------- the calls

class RopePlan(_Plan):
    """A prepared rope(): call it to rotate what x holds then; returns out."""

    def __init__(self, x, rope: Rope, positions, out=None, stream=None):
        import torch

        kind, stride = _rows_view(x, "x")
        t, h, d = x.shape
        _need(positions, "positions", (torch.int32,), shape=(t,))
        _on_current(x, stream)
        if out is None:
            out = _empty((t, h, d), torch.bfloat16, x.device, stream)
        _need(out, "out", (torch.bfloat16,), shape=(t, h, d))
        _, out_stride = _rows_view(out, "out")
        _same_device(x, positions, out, rope.freq)
        self._set(lib().mq_rope, "mq_rope",
                  (ctypes.byref(rope.spec), _ptr(positions), _addr(x), kind, stride, t, h, d,
                   _addr(out), out_stride, _stream(stream)), out, (x, rope, positions, out), t)


def rope(x, rope: Rope, positions, out=None, stream=None):
    """Rotary positions: x bf16 or fp32 [rows, heads, dim] (rows may be parts of
    wider ones), positions int32 [rows] -> bf16 [rows, heads, dim].  out may be
    x itself (bf16)."""
    return RopePlan(x, rope, positions, out, stream)()


class CacheAppendPlan(_Plan):
    """A prepared cache_append(); returns q_out (None without q)."""

    def __init__(self, cache: KVCache, batch: KVBatch, k, v, q=None, rope: Rope = None, q_out=None,
                 stream=None):
        import torch

        kind, stride = _rows_view(k, "k", cache.heads, cache.dim, batch.rows)
        kind_v, stride_v = _rows_view(v, "v", cache.heads, cache.dim, batch.rows)
        if (kind, stride) != (kind_v, stride_v):
            raise ValueError("mq: k and v need one type and one row stride")
        _on_current(k, stream)
        q_stride = q_heads = 0
        if q is not None:
            kind_q, q_stride = _rows_view(q, "q", None, cache.dim, batch.rows)
            if kind_q != kind:
                raise TypeError("mq: q has another type than k and v")
            q_heads = q.shape[1]
            if q_out is None:
                q_out = _empty(tuple(q.shape), torch.bfloat16, q.device, stream)
            _need(q_out, "q_out", (torch.bfloat16,), shape=tuple(q.shape))
            _ptr(q_out)
        elif q_out is not None:
            raise ValueError("mq: q_out without q")
        _same_device(k, v, q, q_out, cache.k, batch.q_start, rope.freq if rope else None)
        self._set(lib().mq_cache_append, "mq_cache_append",
                  (ctypes.byref(cache.c), ctypes.byref(batch.c),
                   ctypes.byref(rope.spec) if rope else None, _addr(k), _addr(v), stride, _addr(q),
                   q_stride, q_heads, kind, _addr(q_out), _stream(stream)), q_out,
                  (cache, batch, k, v, q, rope, q_out), batch.rows)


def cache_append(cache: KVCache, batch: KVBatch, k, v, q=None, rope: Rope = None, q_out=None,
                 stream=None):
    """Quantize the batch's rows of k and v (bf16 or fp32 [rows, heads, dim])
    into the cache; with `rope` k is rotated by its position first.  With q
    [rows, q_heads, dim] the queries are rotated in the same launch and
    returned as bf16."""
    return CacheAppendPlan(cache, batch, k, v, q, rope, q_out, stream)()


def cache_read(cache: KVCache, batch: KVBatch, dtype=None, k_out=None, v_out=None, stream=None):
    """The batch's tokens back from the cache: (k, v) [rows, heads, dim] in
    bf16 (the default) or fp32."""
    import torch

    if dtype is None:
        dtype = torch.bfloat16 if k_out is None else k_out.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("mq: the cache is read as bf16 or fp32")
    shape = (batch.rows, cache.heads, cache.dim)
    _on_current(cache.k, stream)
    if k_out is None:
        k_out = _empty(shape, dtype, cache.k.device, stream)
    if v_out is None:
        v_out = _empty(shape, dtype, cache.k.device, stream)
    _need(k_out, "k_out", (dtype,), shape=shape)
    _need(v_out, "v_out", (dtype,), shape=shape)
    _same_device(cache.k, batch.q_start, k_out, v_out)
    if batch.rows:
        _check(lib().mq_cache_read(ctypes.byref(cache.c), ctypes.byref(batch.c), _ptr(k_out),
                                   _ptr(v_out), _F32 if dtype == torch.float32 else _BF16,
                                   _stream(stream)), "mq_cache_read")
    return k_out, v_out


def cache_attend_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int,
                                 window: int = 0) -> int:
    return int(lib().mq_cache_attend_workspace_bytes(ctypes.byref(cache.c), ctypes.byref(batch.c),
                                                     q_heads, window))


class CacheAttendPlan(_Plan):
    """A prepared cache_attend(); returns out, or (out, lse) if lse was given.
    Its workspace is its own unless one is given."""

    def __init__(self, cache: KVCache, batch: KVBatch, q, scale=None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True, out=None, lse=None, workspace=None,
                 stream=None):
        import torch

        _need(q, "q", (torch.bfloat16,))
        _, stride = _rows_view(q, "q", None, cache.dim, batch.rows)
        t, h, d = q.shape
        _on_current(q, stream)
        if out is None:
            out = _empty((t, h, d), torch.bfloat16, q.device, stream)
        _need(out, "out", (torch.bfloat16,), shape=(t, h, d))
        if lse is not None:
            _need(lse, "lse", (torch.float32,), shape=(t, h))
        need = cache_attend_workspace_bytes(cache, batch, h, window)
        if need and workspace is None:
            workspace = _empty((need,), torch.uint8, q.device, stream)
        if workspace is not None:
            _need(workspace, "workspace", (torch.uint8,))
        _same_device(q, out, lse, workspace, cache.k, batch.q_start)
        ws_bytes = 0 if workspace is None else workspace.numel()
        _ptr(out), _ptr(lse)
        self._set(lib().mq_cache_attend, "mq_cache_attend",
                  (ctypes.byref(cache.c), ctypes.byref(batch.c), _addr(q), stride, h,
                   float(d ** -0.5 if scale is None else scale), float(softcap), int(window),
                   int(bool(causal)), _addr(out), _addr(lse), _ptr(workspace), ws_bytes,
                   _stream(stream)),
                  out if lse is None else (out, lse), (cache, batch, q, out, lse, workspace), t)


def cache_attend(cache: KVCache, batch: KVBatch, q, scale=None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of the batch's queries q bf16 [rows, q_heads, dim] over their
    sequences' cached tokens -> bf16 [rows, q_heads, dim].  scale: dim^-0.5 by
    default; softcap > 0 caps the scores; window > 0: only the last `window`
    tokens up to the query; lse: fp32 [rows, q_heads], filled if given."""
    plan = CacheAttendPlan(cache, batch, q, scale, softcap, window, causal, out, lse, workspace,
                           stream)
    plan()
    return plan.result if lse is None else plan.result[0]


class StackAttention:
    """The attention of a Mix'n'Match stack: one KVCache a layer (same heads,
    dim and block), the batch that its rows belong to, the positions and, per
    layer, a window (0: none)."""

    def __init__(self, caches, batch: KVBatch, q_heads: int, rope: Rope = None, scale=None,
                 softcap: float = 0.0, windows=None):
        self.caches, self.batch, self.rope = list(caches), batch, rope
        if not self.caches:
            raise ValueError("mq: one cache a layer")
        if windows is not None and len(windows) != len(self.caches):
            raise ValueError("mq: one window a layer")
        self.q_heads = int(q_heads)
        _same_device(batch.q_start, rope.freq if rope else None, *(c.k for c in self.caches))
        self._arr = (_Cache * len(self.caches))(*(c.c for c in self.caches))
        self._win = None if windows is None else (ctypes.c_int64 * len(windows))(*windows)
        self.c = _StackAttention(
            self._arr, ctypes.pointer(batch.c), ctypes.pointer(rope.spec) if rope else None,
            self._win, self.q_heads,
            float(self.caches[0].dim ** -0.5 if scale is None else scale), float(softcap))


def mixnmatch_attend_workspace_bytes(layer_arr, attn: StackAttention, M: int) -> int:
    if len(layer_arr) != len(attn.caches):
        raise ValueError("mq: one cache a layer")
    return int(lib().mq_mixnmatch_attend_workspace_bytes(layer_arr, len(layer_arr),
                                                         ctypes.byref(attn.c), M))


def mixnmatch_attend(layer_arr, attn: StackAttention, x=None, h=None, workspace=None, stream=None):
    """Run the stack with attention on bf16 x [M, H] (row m is row m of the
    attention's batch): returns the fp32 residual stream h [M, H].  Without x
    the layers continue the residual stream h, in place."""
    import torch

    if x is None and h is None:
        raise ValueError("mq: x or h is needed")
    m, H = (x if x is not None else h).shape
    width = int(layer_arr[0].q.N) if len(layer_arr) else 0
    if H != width or m != attn.batch.rows:
        raise ValueError(f"mq: the input is [{m}, {H}], expected [{attn.batch.rows}, {width}]")
    dev = (x if x is not None else h).device
    if x is not None:
        _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), shape=(m, H))
    if h is None:
        h = _empty((m, H), torch.float32, dev, stream)
    _need(h, "h", (torch.float32,), shape=(m, H))
    need = mixnmatch_attend_workspace_bytes(layer_arr, attn, m)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, dev, stream)
    _need(workspace, "workspace", (torch.uint8,))
    _same_device(x, h, workspace, attn.batch.q_start)
    _on_current(h, stream)
    _check(lib().mq_mixnmatch_attend(layer_arr, len(layer_arr), ctypes.byref(attn.c), _ptr(x), m,
                                     _ptr(h), _ptr(workspace), workspace.numel(),
                                     _stream(stream)), "mq_mixnmatch_attend")
    return h
