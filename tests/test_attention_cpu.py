"""CPU checks of the attention operators: the oracle against hand-computed and
independent values, the frequencies' scalings, and the refusals of the C ABI
and the Python binding (calls that return before any HIP call)."""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import nested_int_matmul_amd as mq
import oracle
from nested_int_matmul_amd import attention as at

P = 0x10000  # a 16-byte aligned dummy address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mq.LIB_PATH):
        pytest.skip("libmq.so not built")
    return mq.lib()


# ---------------------------------------------------------------- the oracle

def test_e4m3_table_is_the_format():
    t = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, oracle.E4M3)


def test_round_codes_ties_and_saturation():
    x = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.49, 1e9, -1e9, np.nan])
    assert oracle.round_codes(x, "int8").view(np.int8).tolist() == \
        [0, 2, 2, 0, -2, 126, 127, 127, -127, 0]
    # between two neighbours: the one with an even last bit; beyond 448: 448
    e = oracle.E4M3
    mid = (e[:-1] + e[1:]) / 2
    want = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(oracle.round_codes(mid, "e4m3"), want.astype(np.uint8))
    near = np.nextafter(mid, 1e9)
    assert np.array_equal(oracle.round_codes(near, "e4m3"), (np.arange(126) + 1).astype(np.uint8))
    assert oracle.round_codes(np.array([460.0, 1e9, -1e9]), "e4m3").tolist() == [126, 126, 254]
    x = np.random.default_rng(0).standard_normal(4000) * 30
    t = torch.from_numpy(x).float()
    assert np.array_equal(oracle.round_codes(t.double().numpy(), "e4m3"),
                          t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_rope_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 16))
    f = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    pos = np.array([0, 1, 7, 1000, 100000])
    for inter in (False, True):
        y = oracle.rope_turn(x, pos, f, 1.0, inter)
        assert np.allclose((x * x).sum(-1), (y * y).sum(-1))
        assert np.array_equal(y[0], x[0])
        # scores depend on the distance only
        a = oracle.rope_turn(x[:1], np.array([40]), f, 1.0, inter)[0, 0]
        b = oracle.rope_turn(x[1:2], np.array([33]), f, 1.0, inter)[0, 0]
        c = oracle.rope_turn(x[:1], np.array([9]), f, 1.0, inter)[0, 0]
        d = oracle.rope_turn(x[1:2], np.array([2]), f, 1.0, inter)[0, 0]
        assert math.isclose(a @ b, c @ d, rel_tol=1e-9)


def test_oracle_append_grows_and_keeps():
    c = oracle.Cache(np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1, 64, 16), np.uint8),
                     np.zeros((1, 1), np.float32), np.zeros((1, 1), np.float32), "int8")
    one = np.zeros((1, 1, 64))
    one[0, 0, 0] = 127.0
    table = np.zeros((1, 1), np.int32)
    c.append([0, 1], [1], table, one, one)
    assert c.ks[0, 0] == 1.0 and c.k[0, 0, 0, 0] == 127 and c.v[0, 0, 0, 0] == 127
    c.append([0, 1], [2], table, 2 * one, one / 2)
    assert c.ks[0, 0] == 2.0 and c.k[0, 0, :2, 0].tolist() == [64, 127]  # 63.5: to even
    assert c.vs[0, 0] == 1.0 and c.v[0, 0, 0, :2].tolist() == [127, 64]


# ---------------------------------------------------------------- frequencies

def test_rope_frequencies():
    f, m = mq.rope_frequencies(64, base=10000.0, device="cpu")
    i = np.arange(32)
    assert m == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-i / 32), rtol=1e-15)
    g, _ = mq.rope_frequencies(64, scaling={"kind": "linear", "factor": 4}, device="cpu")
    assert np.allclose(g.numpy() * 4, f.numpy(), rtol=1e-15)
    g, _ = mq.rope_frequencies(64, scaling={"kind": "base", "factor": 4}, device="cpu")
    assert math.isclose(g[0], 1.0) and math.isclose(g[31], f[31] / 4, rel_tol=1e-12)
    for kind, high in (("bands", 4.0), ("yarn", 32.0)):
        g, m = mq.rope_frequencies(64, scaling={"kind": kind, "factor": 8, "trained": 4096},
                                   device="cpu")
        turns = 4096 * f.numpy() / (2 * math.pi)
        assert np.array_equal(g.numpy()[turns >= high], f.numpy()[turns >= high])
        assert np.allclose(g.numpy()[turns <= 1] * 8, f.numpy()[turns <= 1], rtol=1e-15)
        assert np.all(np.diff(g.numpy()) < 0)
        assert math.isclose(m, 1.0 if kind == "bands" else 0.1 * math.log(8) + 1)
    for bad in ({"kind": "linear"}, {"kind": "x", "factor": 2}, {"kind": "yarn", "factor": 2},
                {"kind": "bands", "factor": 2, "trained": 10, "low": 4, "high": 4}):
        with pytest.raises(ValueError):
            mq.rope_frequencies(64, scaling=bad, device="cpu")
    for rot in (0, 4, 12):
        with pytest.raises(ValueError):
            mq.rope_frequencies(rot, device="cpu")


# ---------------------------------------------------------------- C ABI refusals

def _cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, pages=10, heads=8, block=64, dim=128, format=0)
    d.update(kw)
    return at._Cache(**d)


def _batch(**kw):
    d = dict(q_start=P, kv_len=P, page_table=P, rows=4, seqs=4, table_pages=8, max_new=1)
    d.update(kw)
    return at._Batch(**d)


def _rope(**kw):
    d = dict(freq=P, factor=1.0, rot=128, interleaved=0)
    d.update(kw)
    return at._RopeSpec(**d)


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
             (dict(v_scale=None), 1), (dict(format=2), 3), (dict(format=-1), 3),
             (dict(pages=0), 2), (dict(pages=1 << 31), 2), (dict(heads=0), 2),
             (dict(heads=4097), 2), (dict(block=8), 2), (dict(block=48), 2), (dict(block=256), 2),
             (dict(dim=96), 2), (dict(dim=0), 2), (dict(dim=512), 2), (dict(k=P + 8), 5),
             (dict(v=P + 1), 5), (dict(k_scale=P + 2), 5), (dict(v_scale=P + 1), 5)]
BAD_BATCH = [(dict(q_start=None), 1), (dict(kv_len=None), 1), (dict(page_table=None), 1),
             (dict(rows=-1), 2), (dict(rows=1 << 31), 2), (dict(seqs=0), 2),
             (dict(seqs=65536), 2), (dict(table_pages=0), 2), (dict(table_pages=1 << 25), 2),
             (dict(table_pages=-5), 2), (dict(max_new=0), 2), (dict(max_new=(1 << 24) + 1), 2),
             (dict(q_start=P + 1), 5), (dict(kv_len=P + 2), 5), (dict(page_table=P + 3), 5)]
BAD_ROPE = [(dict(freq=None), 1), (dict(freq=P + 4), 5), (dict(rot=0), 2), (dict(rot=-8), 2),
            (dict(rot=12), 2), (dict(rot=136), 2), (dict(interleaved=2), 3),
            (dict(factor=math.inf), 3), (dict(factor=math.nan), 3)]


def _append(L, c=None, b=None, r=None, k=P, v=P, ks=1024, q=None, qs=4096, qh=32, t=0, qo=None):
    ref = lambda x: ctypes.byref(x) if x is not None else None  # noqa: E731
    return L.mq_cache_append(ref(c or _cache()), ref(b or _batch()), ref(r), k, v, ks, q, qs, qh,
                             t, qo, None)


def _attend(L, c=None, b=None, q=P, qs=4096, qh=32, scale=0.1, cap=0.0, win=0, causal=1, out=P,
            lse=None, ws=P, wb=1 << 40):
    return L.mq_cache_attend(ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), q, qs, qh,
                             scale, cap, win, causal, out, lse, ws, wb, None)


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches(L, kw, want):
    c = _cache(**kw)
    assert _append(L, c=c) == want
    assert L.mq_cache_read(ctypes.byref(c), ctypes.byref(_batch()), P, P, 0, None) == want
    assert _attend(L, c=c) == want
    assert L.mq_cache_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(_batch()), 32, 0) == 0


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_bad_batches(L, kw, want):
    b = _batch(**kw)
    assert _append(L, b=b) == want
    assert L.mq_cache_read(ctypes.byref(_cache()), ctypes.byref(b), P, P, 0, None) == want
    assert _attend(L, b=b) == want
    assert L.mq_cache_attend_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(b), 32, 0) == 0


@pytest.mark.parametrize("kw,want", BAD_ROPE)
def test_bad_rope(L, kw, want):
    r = _rope(**kw)
    assert _append(L, r=r) == want
    assert L.mq_rope(ctypes.byref(r), P, P, 0, 1024, 4, 8, 128, P, 1024, None) == want


def test_null_structs(L):
    assert L.mq_cache_append(None, ctypes.byref(_batch()), None, P, P, 1024, None, 0, 0, 0, None,
                             None) == 1
    assert L.mq_cache_read(ctypes.byref(_cache()), None, P, P, 0, None) == 1
    assert L.mq_rope(None, P, P, 0, 1024, 4, 8, 128, P, 1024, None) == 1
    assert L.mq_cache_attend(None, None, P, 4096, 32, 1.0, 0.0, 0, 1, P, None, P, 1 << 40,
                             None) == 1
    assert L.mq_cache_attend_workspace_bytes(None, None, 32, 0) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=P), 1), (dict(qo=P), 1), (dict(t=2), 3),
    (dict(t=-1), 3), (dict(ks=1016), 2), (dict(ks=1028), 5), (dict(ks=1 << 41), 2),
    (dict(k=P + 8), 5), (dict(v=P + 2), 5), (dict(q=P, qo=P, qh=0), 2),
    (dict(q=P, qo=P, qs=4088), 2), (dict(q=P, qo=P, qs=4100), 5), (dict(q=P + 4, qo=P), 5),
    (dict(q=P, qo=P + 8), 5), (dict(q=P, qo=P, qh=1 << 20), 2)])
def test_append_refusals(L, kw, want):
    assert _append(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(qh=12), 2), (dict(qh=0), 2),
    (dict(qh=1 << 14), 2), (dict(qs=4088), 2), (dict(qs=4097), 5), (dict(q=P + 8), 5),
    (dict(out=P + 2), 5), (dict(lse=P + 2), 5), (dict(scale=math.nan), 3),
    (dict(scale=math.inf), 3), (dict(cap=-1.0), 3), (dict(cap=math.inf), 3),
    (dict(cap=1e-35), 3), (dict(win=-1), 2), (dict(win=5, causal=0), 2), (dict(causal=2), 3),
    (dict(b=_batch(max_new=1 << 22)), 2), (dict(b=_batch(rows=1 << 28)), 2)])
def test_attend_refusals(L, kw, want):
    assert _attend(L, **kw) == want


def test_attend_most_rows(L):
    """Rows times query heads up to 2^25, the largest grid."""
    c = _cache()
    most, more = (_batch(rows=n, table_pages=512) for n in (1 << 20, (1 << 20) + 1))
    bytes_of = L.mq_cache_attend_workspace_bytes
    assert bytes_of(ctypes.byref(c), ctypes.byref(most), 32, 0) > 0
    assert bytes_of(ctypes.byref(c), ctypes.byref(more), 32, 0) == 0
    assert _attend(L, b=more) == 2


def test_attend_workspace(L):
    c, b = _cache(), _batch(seqs=2, rows=2, table_pages=512)
    need = L.mq_cache_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 32, 0)
    assert need > 0
    assert _attend(L, b=b, ws=None, wb=0) == 6
    assert _attend(L, b=b, wb=need - 1) == 6
    assert _attend(L, b=b, ws=P + 16, wb=need) == 5
    # a window bounds the keys, and with them the pieces
    small = L.mq_cache_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 32, 64)
    assert small < need
    huge = L.mq_cache_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 32, (1 << 63) - 1)
    assert huge == need


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(t=5), 3),
    (dict(rows=-1), 2), (dict(rows=(1 << 24) + 1), 2), (dict(heads=0), 2), (dict(dim=132), 2),
    (dict(dim=0), 2), (dict(dim=1032), 2), (dict(heads=1 << 20), 2), (dict(xs=1016), 2),
    (dict(os=1016), 2), (dict(xs=1028), 5), (dict(os=1028), 5), (dict(x=P + 4), 5),
    (dict(out=P + 4), 5), (dict(pos=P + 2), 5), (dict(out=P, t=1), 2), (dict(out=P, os=2048), 2)])
def test_rope_refusals(L, kw, want):
    d = dict(pos=P, x=P, t=0, xs=1024, rows=4, heads=8, dim=128, out=2 * P, os=1024)
    d.update(kw)
    assert L.mq_rope(ctypes.byref(_rope(rot=8)), d["pos"], d["x"], d["t"], d["xs"], d["rows"],
                     d["heads"], d["dim"], d["out"], d["os"], None) == want


def test_read_refusals(L):
    c, b = ctypes.byref(_cache()), ctypes.byref(_batch())
    assert L.mq_cache_read(c, b, None, None, 0, None) == 1
    assert L.mq_cache_read(c, b, P, P, 2, None) == 3
    assert L.mq_cache_read(c, b, P + 8, P, 0, None) == 5
    assert L.mq_cache_read(c, b, None, P + 2, 0, None) == 5


# ---------------------------------------------------------------- Python refusals

def test_python_refusals_without_a_gpu():
    with pytest.raises(TypeError):
        mq.Rope(torch.zeros(8))
    k = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    v = torch.zeros((2, 1, 64, 16), dtype=torch.uint8)
    s = torch.zeros((2, 1))
    with pytest.raises(ValueError):
        mq.KVCache(k, v, s, s, "int4")
    with pytest.raises(ValueError):
        mq.KVCache(k, k, s, s, "int8")
    with pytest.raises(ValueError):
        mq.KVCache(k, v, s[:1], s, "int8")
    with pytest.raises(TypeError):
        mq.KVCache(k, v, s.double(), s, "int8")
    with pytest.raises(ValueError):  # not on the GPU
        mq.KVCache(k, v, s, s, "int8")
    i = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        mq.KVBatch(i.long(), i[:2], table, 2, 1)
    with pytest.raises(ValueError):
        mq.KVBatch(i, i, table, 2, 1)
    with pytest.raises(ValueError):
        mq.KVBatch(i, i[:2], table[0], 2, 1)
    with pytest.raises(ValueError):
        mq.KVBatch(i, i[:2], table, -1, 1)
