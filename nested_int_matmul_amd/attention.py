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
A plan uses the tensors it was made of at their addresses, keeps them alive and
launches on the stream that was current when it was made (or the one given).
Calls must be made with the tensors' device as the current device.
"""

from __future__ import annotations

import ctypes
import math

from . import MQ_OK, MQError, _need, lib

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
#
# A decode step makes these calls at the rate of launches, so each tensor is
# looked at once and addresses go to ctypes as plain integers.

def _address(t, name, dtypes, device, shape=None):
    """Address of a contiguous tensor on `device` of one of the types."""
    _need(t, name, dtypes, shape=shape)
    if t.device != device:
        if not t.is_cuda:
            raise ValueError("mq: tensors must be on the GPU")
        raise ValueError(f"mq: {name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"mq: {name} must be contiguous (row-major)")
    return t.data_ptr()


def _current_stream(index):
    """Address of the current stream of a device (without making a Stream
    object, where torch offers that: 0.1 against 2.8 us)."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw else torch.cuda.current_stream(index).cuda_stream


def _launch_on(t, stream):
    """Address of the stream to launch on.  Work is launched on the current
    device: the tensors have to be there, and a stream given has to be its."""
    import torch

    if not t.is_cuda:
        raise ValueError("mq: tensors must be on the GPU")
    index = t.get_device()
    if index != torch.cuda.current_device():
        raise ValueError(f"mq: tensors on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return _current_stream(index)
    if stream.device != t.device:
        raise ValueError(f"mq: a stream of {stream.device} for tensors on {t.device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A tensor that the call writes, from the memory of the stream it runs on
    (so that its memory is reused in that stream's order)."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(t, name, dtype, device, shape, stream):
    """The tensor that the call writes and its address: the given one, checked,
    or a new one."""
    if t is None:
        t = _empty(shape, dtype, device, stream)
        return t, t.data_ptr()
    return t, _address(t, name, (dtype,), device, shape)


def _rows_view(x, name, device, heads=None, dim=None, rows=None):
    """x bf16 or fp32 [rows, heads, dim] on `device` whose rows are contiguous
    and evenly spaced (it may be a part of wider rows): (type, row stride in
    entries, address)."""
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError(f"mq: {name} must be a tensor")
    kind = _F32 if x.dtype is torch.float32 else _BF16
    if kind == _BF16 and x.dtype is not torch.bfloat16:
        raise TypeError(f"mq: {name} has dtype {x.dtype}, expected bfloat16 or float32")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"mq: {name} must be [rows, heads, dim]")
    if x.device != device:
        if not x.is_cuda:
            raise ValueError("mq: tensors must be on the GPU")
        raise ValueError(f"mq: {name} is on {x.device}, expected {device}")
    t, h, d = shape
    if (heads is not None and h != heads) or (dim is not None and d != dim) or \
            (rows is not None and t != rows):
        want = tuple("any" if v is None else v for v in (rows, heads, dim))
        raise ValueError(f"mq: {name} has shape {tuple(shape)}, expected {want}")
    s0, s1, s2 = x.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"mq: the rows of {name} must be contiguous")
    if t <= 1:
        s0 = h * d
    elif s0 < h * d:
        raise ValueError(f"mq: the rows of {name} overlap")
    return kind, s0, x.data_ptr()


def _run(fn, name, args, rows):
    if rows:  # (no rows: nothing to do, and empty tensors have no address)
        st = fn(*args)
        if st != MQ_OK:
            raise MQError(st, name)


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
        if not freq.is_cuda:
            raise ValueError("mq: tensors must be on the GPU")
        self.spec = _RopeSpec(_address(freq, "freq", (torch.float64,), freq.device), self.factor,
                              self.rot, int(self.interleaved))
        self.device, self.ref = freq.device, ctypes.byref(self.spec)


class KVCache:
    """A paged 8-bit cache of one layer: k uint8 [pages, heads, block, dim],
    v uint8 [pages, heads, dim, block] (dim-major), k_scale and v_scale fp32
    [pages, heads]; value = code * scale; fmt "int8" or "e4m3"."""

    def __init__(self, k, v, k_scale, v_scale, fmt: str):
        import torch

        _need(k, "k", (torch.uint8,))
        if k.dim() != 4:
            raise ValueError("mq: k must be [pages, heads, block, dim]")
        p, h, b, d = k.shape
        dev = k.device
        if fmt not in KV_FORMATS:
            raise ValueError(f"mq: unknown cache format {fmt!r}")
        _need(v, "v", (torch.uint8,), shape=(p, h, d, b))
        _need(k_scale, "k_scale", (torch.float32,), shape=(p, h))
        _need(v_scale, "v_scale", (torch.float32,), shape=(p, h))
        if not k.is_cuda:
            raise ValueError("mq: tensors must be on the GPU")
        self.k, self.v, self.k_scale, self.v_scale, self.fmt = k, v, k_scale, v_scale, fmt
        self.pages, self.heads, self.block, self.dim, self.device = p, h, b, d, dev
        self.c = _Cache(_address(k, "k", (torch.uint8,), dev),
                        _address(v, "v", (torch.uint8,), dev),
                        _address(k_scale, "k_scale", (torch.float32,), dev),
                        _address(v_scale, "v_scale", (torch.float32,), dev), p, h, b, d,
                        KV_FORMATS[fmt])
        self.ref = ctypes.byref(self.c)

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
        dev = q_start.device
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.rows, self.max_new, self.seqs = int(rows), int(max_new), s
        if not (0 <= self.rows < 1 << 31 and 1 <= self.max_new < 1 << 31):
            raise ValueError("mq: rows or max_new out of range")
        if not q_start.is_cuda:
            raise ValueError("mq: tensors must be on the GPU")
        self.device = dev
        self.c = _Batch(_address(q_start, "q_start", i32, dev),
                        _address(kv_len, "kv_len", i32, dev),
                        _address(page_table, "page_table", i32, dev), self.rows, s, wide,
                        self.max_new)
        self.ref = ctypes.byref(self.c)


class _Plan:
    """A checked and marshalled call: calling it makes the C call and returns
    `result`.  `keep`: what the addresses belong to."""

    def __init__(self, fn, name, args, rows, result, keep):
        self.fn, self.name, self.args, self.rows = fn, name, args, rows
        self.result, self.keep = result, keep

    def __call__(self):
        _run(self.fn, self.name, self.args, self.rows)
        return self.result


def _one_device(device, *others):
    for o in others:
        if o is not None and o.device != device:
            raise ValueError(f"mq: tensors on different devices: {device} and {o.device}")


# ---------------------------------------------------------------- the calls

def _rope_call(x, rope, positions, out, stream):
    import torch

    at = _launch_on(x, stream)
    dev = x.device
    kind, stride, px = _rows_view(x, "x", dev)
    t, h, d = x.shape
    pp = _address(positions, "positions", (torch.int32,), dev, (t,))
    _one_device(dev, rope)
    if out is None:
        out = _empty((t, h, d), torch.bfloat16, dev, stream)
    kind_out, out_stride, po = _rows_view(out, "out", dev, h, d, t)
    if kind_out != _BF16:
        raise TypeError("mq: out must be bf16")
    return (rope.ref, pp, px, kind, stride, t, h, d, po, out_stride, at), t, out


def rope(x, rope: Rope, positions, out=None, stream=None):
    """Rotary positions: x bf16 or fp32 [rows, heads, dim] (rows may be parts of
    wider ones), positions int32 [rows] -> bf16 [rows, heads, dim].  out may be
    x itself (bf16)."""
    args, t, out = _rope_call(x, rope, positions, out, stream)
    _run(lib().mq_rope, "mq_rope", args, t)
    return out


class RopePlan(_Plan):
    """A prepared rope(): call it to rotate what x holds then; returns out."""

    def __init__(self, x, rope: Rope, positions, out=None, stream=None):
        args, t, out = _rope_call(x, rope, positions, out, stream)
        super().__init__(lib().mq_rope, "mq_rope", args, t, out, (x, rope, positions))


def _append_call(cache, batch, k, v, q, rope, q_out, stream):
    import torch

    at = _launch_on(k, stream)
    dev = k.device
    rows, dim = batch.rows, cache.dim
    kind, stride, pk = _rows_view(k, "k", dev, cache.heads, dim, rows)
    kind_v, stride_v, pv = _rows_view(v, "v", dev, cache.heads, dim, rows)
    if (kind, stride) != (kind_v, stride_v):
        raise ValueError("mq: k and v need one type and one row stride")
    _one_device(dev, cache, batch, rope)
    q_stride, q_heads, pq, po = 0, 0, None, None
    if q is not None:
        kind_q, q_stride, pq = _rows_view(q, "q", dev, None, dim, rows)
        if kind_q != kind:
            raise TypeError("mq: q has another type than k and v")
        shape = tuple(q.shape)
        q_heads = shape[1]
        q_out, po = _output(q_out, "q_out", torch.bfloat16, dev, shape, stream)
    elif q_out is not None:
        raise ValueError("mq: q_out without q")
    return (cache.ref, batch.ref, rope.ref if rope is not None else None, pk, pv, stride, pq,
            q_stride, q_heads, kind, po, at), rows, q_out


def cache_append(cache: KVCache, batch: KVBatch, k, v, q=None, rope: Rope = None, q_out=None,
                 stream=None):
    """Quantize the batch's rows of k and v (bf16 or fp32 [rows, heads, dim])
    into the cache; with `rope` k is rotated by its position first.  With q
    [rows, q_heads, dim] the queries are rotated in the same launch and
    returned as bf16 (in q_out)."""
    args, rows, q_out = _append_call(cache, batch, k, v, q, rope, q_out, stream)
    _run(lib().mq_cache_append, "mq_cache_append", args, rows)
    return q_out


class CacheAppendPlan(_Plan):
    """A prepared cache_append(); returns q_out (None without q)."""

    def __init__(self, cache: KVCache, batch: KVBatch, k, v, q=None, rope: Rope = None, q_out=None,
                 stream=None):
        args, rows, q_out = _append_call(cache, batch, k, v, q, rope, q_out, stream)
        super().__init__(lib().mq_cache_append, "mq_cache_append", args, rows, q_out,
                         (cache, batch, k, v, q, rope))


def cache_read(cache: KVCache, batch: KVBatch, dtype=None, k_out=None, v_out=None, stream=None):
    """The batch's tokens back from the cache: (k, v) [rows, heads, dim] in
    bf16 (the default) or fp32."""
    import torch

    if dtype is None:
        dtype = torch.bfloat16 if k_out is None else k_out.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("mq: the cache is read as bf16 or fp32")
    at = _launch_on(cache.k, stream)
    dev = cache.device
    _one_device(dev, batch)
    shape = (batch.rows, cache.heads, cache.dim)
    k_out, pk = _output(k_out, "k_out", dtype, dev, shape, stream)
    v_out, pv = _output(v_out, "v_out", dtype, dev, shape, stream)
    args = (cache.ref, batch.ref, pk, pv, _F32 if dtype is torch.float32 else _BF16, at)
    _run(lib().mq_cache_read, "mq_cache_read", args, batch.rows)
    return k_out, v_out


def cache_attend_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int,
                                 window: int = 0) -> int:
    return int(lib().mq_cache_attend_workspace_bytes(cache.ref, batch.ref, q_heads, window))


def _attend_call(cache, batch, q, scale, softcap, window, causal, out, lse, workspace, stream):
    import torch

    at = _launch_on(q, stream)
    dev = q.device
    kind, stride, pq = _rows_view(q, "q", dev, None, cache.dim, batch.rows)
    if kind != _BF16:
        raise TypeError("mq: q must be bf16")
    _one_device(dev, cache, batch)
    t, h, d = q.shape
    out, po = _output(out, "out", torch.bfloat16, dev, (t, h, d), stream)
    pl = None if lse is None else _address(lse, "lse", (torch.float32,), dev, (t, h))
    pw, nw = None, 0
    if workspace is not None:
        pw, nw = _address(workspace, "workspace", (torch.uint8,), dev), workspace.numel()
    else:
        nw = cache_attend_workspace_bytes(cache, batch, h, window)
        if nw:
            workspace = _empty((nw,), torch.uint8, dev, stream)
            pw = workspace.data_ptr()
    return (cache.ref, batch.ref, pq, stride, h, d ** -0.5 if scale is None else scale, softcap,
            window, 1 if causal else 0, po, pl, pw, nw, at), t, out, workspace


def cache_attend(cache: KVCache, batch: KVBatch, q, scale=None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of the batch's queries q bf16 [rows, q_heads, dim] over their
    sequences' cached tokens -> bf16 [rows, q_heads, dim].  scale: dim^-0.5 by
    default; softcap > 0 caps the scores; window > 0: only the last `window`
    tokens up to the query; lse: fp32 [rows, q_heads], filled if given."""
    args, t, out, _ = _attend_call(cache, batch, q, scale, softcap, window, causal, out, lse,
                                   workspace, stream)
    _run(lib().mq_cache_attend, "mq_cache_attend", args, t)
    return out


class CacheAttendPlan(_Plan):
    """A prepared cache_attend(); returns out, or (out, lse) if lse was given.
    Its workspace is its own unless one is given."""

    def __init__(self, cache: KVCache, batch: KVBatch, q, scale=None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True, out=None, lse=None, workspace=None,
                 stream=None):
        args, t, out, workspace = _attend_call(cache, batch, q, scale, softcap, window, causal, out,
                                               lse, workspace, stream)
        super().__init__(lib().mq_cache_attend, "mq_cache_attend", args, t,
                         out if lse is None else (out, lse), (cache, batch, q, workspace))


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
        _one_device(batch.device, rope, *self.caches)
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
    first = x if x is not None else h
    at, dev = _launch_on(first, stream), first.device
    _one_device(dev, attn.batch)
    px = None
    if x is not None:
        px = _address(x, "x", (torch.bfloat16, torch.int16, torch.uint16), dev, (m, H))
    h, ph = _output(h, "h", torch.float32, dev, (m, H), stream)
    if workspace is None:
        need = mixnmatch_attend_workspace_bytes(layer_arr, attn, m)
        workspace = _empty((max(need, 1),), torch.uint8, dev, stream)
    pw = _address(workspace, "workspace", (torch.uint8,), dev)
    if len(layer_arr) != len(attn.caches):
        raise ValueError("mq: one cache a layer")
    _run(lib().mq_mixnmatch_attend, "mq_mixnmatch_attend",
         (layer_arr, len(layer_arr), ctypes.byref(attn.c), px, m, ph, pw, workspace.numel(), at), 1)
    return h
