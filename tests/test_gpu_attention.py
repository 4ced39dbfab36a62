"""GPU tests of the rotary positions, the 8-bit cache and the attention over it
against the float64 oracle: codes and scales byte for byte, results within
bounds derived from the arithmetic (attention_helpers.attend_bounds)."""

import numpy as np
import pytest
import torch

import nested_int_matmul_amd as mq
import oracle
from attention_helpers import (assert_attend, assert_cache_equal, bf16_values, device, device_batch,
                               device_bf16, device_cache, filled, make_table, stale_cache, starts)

pytestmark = pytest.mark.gpu


def _freq(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot)


def _rope(rot, factor=1.0, interleaved=False, freq=None):
    f = _freq(rot) if freq is None else freq
    return mq.Rope(device(np.asarray(f, np.float64)), factor, interleaved)


def _bits(t):
    return t.cpu().view(torch.int16).numpy()


def _same_bf16(got, want, what=""):
    """bf16 tensor against bf16 values in float64, bit for bit (zeros of either sign)."""
    g = got.double().cpu().numpy()
    bad = g != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} entries differ"


# ---------------------------------------------------------------- rope

@pytest.mark.parametrize("rows,heads,dim,rot,inter,kind,wide", [
    (1, 1, 64, 64, False, "bf16", False),
    (8, 32, 128, 128, False, "fp32", False),
    (3, 5, 128, 64, True, "fp32", True),
    (17, 7, 256, 64, False, "bf16", True),
    (33, 2, 80, 40, False, "fp32", False),
    (5, 3, 96, 24, True, "bf16", False),
    (2, 1, 8, 8, False, "fp32", False),
    (129, 1, 1024, 1024, True, "bf16", False),
    (3000, 4, 64, 64, False, "bf16", False),
])
def test_rope(rows, heads, dim, rot, inter, kind, wide):
    rng = np.random.default_rng(rows * 31 + dim)
    full = bf16_values(rng, (rows, heads + (3 if wide else 0), dim)) if kind == "bf16" else \
        rng.standard_normal((rows, heads + (3 if wide else 0), dim)).astype(np.float32)
    pos = rng.integers(0, 200000, rows).astype(np.int32)
    x = device(np.asarray(full, np.float32)).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    x = x[:, :heads]
    got = mq.rope(x, _rope(rot, 1.25, inter), device(pos))
    want = oracle.to_bf16(oracle.rope_turn(full[:, :heads], pos, _freq(rot), 1.25, inter))
    _same_bf16(got, want)


def test_rope_far_positions_and_in_place():
    rng = np.random.default_rng(5)
    x = bf16_values(rng, (6, 2, 64))
    pos = np.array([2 ** 31 - 1, 2 ** 30 + 1, 16777217, 0, 1, 131071], dtype=np.int32)
    want = oracle.to_bf16(oracle.rope_turn(x, pos, _freq(64)))
    t = device_bf16(x)
    assert mq.rope(t, _rope(64), device(pos), out=t) is t
    _same_bf16(t, want)


def test_rope_no_rows_and_guard():
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert mq.rope(e, _rope(64), device(np.zeros(0, np.int32))).shape == (0, 4, 64)
    # an output inside a larger buffer: nothing around its rows changes
    buf = torch.full((7, 6 * 64), 3.5, dtype=torch.bfloat16, device="cuda")
    out = buf.view(7, 6, 64)[1:6, 1:3]
    x = bf16_values(np.random.default_rng(2), (5, 2, 64))
    pos = np.arange(5, dtype=np.int32)
    mq.rope(device_bf16(x), _rope(64), device(pos), out=out)
    _same_bf16(out, oracle.to_bf16(oracle.rope_turn(x, pos, _freq(64))))
    rest = buf.view(7, 6, 64).clone()
    rest[1:6, 1:3] = 3.5
    assert torch.all(rest == 3.5)


def test_rope_special_values():
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :6] = [np.inf, np.nan, 3e38, 1e-40, -0.0, 1.0]
    got = mq.rope(device(x), _rope(8), device(np.array([3], np.int32))).float().cpu().numpy()[0, 0]
    # pairs (i, i + 4), i < 4: infinity and NaN stay in their pairs
    assert not np.isfinite(got[[0, 4]]).any() and np.isnan(got[[1, 5]]).all()
    assert np.isfinite(got[[2, 3, 6, 7]]).all() and np.all(got[8:] == 0)


# ---------------------------------------------------------------- append and read

def _append_case(seed, lens0, new, heads, block, dim, fmt, kind="bf16", rot=0, q_heads=0,
                 inter=False, spread=6.0):
    """Sequences of lens0 tokens get `new` more; returns everything checked."""
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(lens0, new)]
    pages, table = make_table(rng, lens, block)
    c = stale_cache(rng, pages, heads, block, dim, fmt)
    at0 = starts(lens0)
    c.append(at0, np.asarray(lens0), table, bf16_values(rng, (int(at0[-1]), heads, dim)),
             bf16_values(rng, (int(at0[-1]), heads, dim), 1.0))
    dev = device_cache(c)
    at = starts(new)
    t = int(at[-1])
    wide = rng.standard_normal((t, q_heads + 2 * heads, dim)) * spread
    wide = oracle.to_bf16(wide) if kind == "bf16" else wide.astype(np.float32).astype(np.float64)
    x = device(wide.astype(np.float32)).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    q = x[:, :q_heads] if q_heads else None
    k, v = x[:, q_heads:q_heads + heads], x[:, q_heads + heads:]
    batch = device_batch(at, lens, table)
    rope = _rope(rot, 1.0, inter) if rot else None
    got_q = mq.cache_append(dev, batch, k, v, q=q, rope=rope)
    pos = np.concatenate([np.arange(a, b) for a, b in zip(lens0, lens)]) if t else np.zeros(0)
    turn = (lambda y: oracle.rope_turn(y, pos, _freq(rot), 1.0, inter)) if rot else (lambda y: y)
    kk = oracle.to_bf16(turn(wide[:, q_heads:q_heads + heads]))
    c.append(at, np.asarray(lens), table, kk, oracle.to_bf16(wide[:, q_heads + heads:]))
    assert_cache_equal(dev, c)
    if q_heads:
        _same_bf16(got_q, oracle.to_bf16(turn(wide[:, :q_heads])), "q")
    else:
        assert got_q is None
    return c, dev, table, lens


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block,dim", [(16, 64), (32, 64), (64, 64), (128, 64), (16, 128),
                                       (32, 128), (64, 128), (128, 128), (16, 256), (32, 256),
                                       (64, 256), (128, 256)])
def test_append_and_read(block, dim, fmt):
    lens0 = [0, 5, block - 1, 2 * block + 7, 0, block]
    new = [2 * block + 3, 1, 1, 20, 0, 17]
    c, dev, table, lens = _append_case(block + dim, lens0, new, 2, block, dim, fmt)
    at = starts(lens)
    batch = device_batch(at, lens, table)
    k, v = mq.cache_read(dev, batch, dtype=torch.float32)
    rk, rv = c.read(at, lens, table, int(at[-1]))
    # one fp32 product: its rounding is the float64 product's
    assert np.array_equal(k.cpu().numpy(), rk.astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), rv.astype(np.float32))
    k, v = mq.cache_read(dev, batch)
    _same_bf16(k, oracle.to_bf16(rk))
    _same_bf16(v, oracle.to_bf16(rv))
    # the last tokens only
    some = [min(3, x) for x in lens]
    k, v = mq.cache_read(dev, device_batch(starts(some), lens, table), dtype=torch.float32)
    rk, rv = c.read(starts(some), lens, table, sum(some))
    assert np.array_equal(k.cpu().numpy(), rk.astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), rv.astype(np.float32))


@pytest.mark.parametrize("kind,rot,q_heads,inter,heads,dim,block,fmt", [
    ("fp32", 128, 8, False, 2, 128, 64, "int8"),
    ("bf16", 64, 3, True, 3, 128, 32, "e4m3"),
    ("fp32", 24, 0, False, 1, 64, 16, "e4m3"),
    ("bf16", 256, 5, False, 1, 256, 128, "int8"),
    ("bf16", 0, 40, False, 2, 64, 64, "int8"),
    ("fp32", 16, 33, True, 1, 256, 16, "int8"),
])
def test_append_with_rotation_and_queries(kind, rot, q_heads, inter, heads, dim, block, fmt):
    _append_case(rot + dim, [3, 0, 200, block], [1, 2 * block + 9, 30, 1], heads, block, dim, fmt,
                 kind, rot, q_heads, inter)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token(fmt):
    """Forty decode steps of three sequences, the scales growing on the way."""
    rng = np.random.default_rng(9)
    heads, block, dim, steps = 2, 16, 64, 40
    first = [0, 7, 30]
    pages, table = make_table(rng, [x + steps for x in first], block)
    c = stale_cache(rng, pages, heads, block, dim, fmt)
    at0 = starts(first)
    c.append(at0, first, table, *(bf16_values(rng, (int(at0[-1]), heads, dim)) for _ in range(2)))
    dev = device_cache(c)
    lens = device(np.asarray(first, np.int32))
    kx = torch.empty((3, heads, dim), dtype=torch.bfloat16, device="cuda")
    vx = torch.empty_like(kx)
    batch = mq.KVBatch(device(starts([1, 1, 1])), lens, device(table), rows=3, max_new=1)
    plan = mq.CacheAppendPlan(dev, batch, kx, vx)
    for i in range(steps):
        grow = 1.15 ** i
        k, v = (oracle.to_bf16(rng.standard_normal((3, heads, dim)) * grow) for _ in range(2))
        kx.copy_(device_bf16(k))
        vx.copy_(device_bf16(v))
        lens += 1
        plan()
        c.append(starts([1, 1, 1]), [x + i + 1 for x in first], table, k, v)
        assert_cache_equal(dev, c, f"step {i}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_zeros_infinities_nan_and_tiny(fmt):
    rng = np.random.default_rng(4)
    heads, block, dim = 1, 32, 64
    lens = [32, 32, 32, 32, 32]
    pages, table = make_table(rng, lens, block)
    c = stale_cache(rng, pages, heads, block, dim, fmt)
    dev = device_cache(c)
    k = oracle.to_bf16(rng.standard_normal((160, heads, dim)))
    k[0:32] = 0.0
    k[33, 0, 3], k[34, 0, 4], k[35, 0, 5] = np.inf, -np.inf, np.nan
    k[64:96] = np.where(rng.random((32, heads, dim)) < 0.5, np.inf, np.nan)
    k[96:128] = oracle.to_bf16(k[96:128] * 2.0 ** -97)   # below the smallest scale
    k[128:160] = oracle.to_bf16(k[128:160] * 2.0 ** 125)  # near the largest numbers
    k[128, 0, 0] = 3.3895313892515355e38
    v = k[::-1].copy()
    batch = device_batch(starts(lens), lens, table)
    mq.cache_append(dev, batch, device_bf16(k), device_bf16(v))
    c.append(starts(lens), lens, table, k, v)
    assert_cache_equal(dev, c)


def test_quotients_next_to_borders():
    """Every bf16 mantissa against scales whose quotients fall on and beside the
    borders between codes."""
    rng = np.random.default_rng(12)
    block, dim = 128, 256
    for fmt in ("int8", "e4m3"):
        pages = 64
        table = np.arange(pages, dtype=np.int32)[:, None]
        c = oracle.Cache(np.zeros((pages, 1, block, dim), np.uint8),
                         np.zeros((pages, 1, dim, block), np.uint8),
                         np.zeros((pages, 1), np.float32), np.zeros((pages, 1), np.float32), fmt)
        dev = device_cache(c)
        amax = oracle.to_bf16(1.0 + rng.integers(0, 128, pages) / 128)
        j = np.arange(block * dim) % 2048
        k = np.empty((pages, block, dim))
        for p in range(pages):
            # every mantissa over nine binades below amax, both signs
            x = (1 + (j % 128) / 128) * 2.0 ** -(j // 128 % 9) * np.where(j < 1152, 1, -1)
            x = np.where(np.abs(x) > amax[p], amax[p] / 2, x)
            x[0] = amax[p]
            k[p] = oracle.to_bf16(x).reshape(block, dim)
        k = k.reshape(pages * block, 1, dim)
        lens = [block] * pages
        mq.cache_append(dev, device_batch(starts(lens), lens, table), device_bf16(k), device_bf16(-k))
        c.append(starts(lens), lens, table, k, -k)
        assert_cache_equal(dev, c, fmt)


def test_bad_pages_and_positions_are_left_alone():
    """Page entries outside the pool, positions beyond the table and before 0,
    rows beyond the last sequence: nothing there is written, the rest is."""
    rng = np.random.default_rng(6)
    heads, block, dim = 2, 16, 64
    lens, new = [40, 40, 70, 3, 24], [40, 20, 70, 5, 24]
    table = np.array([[0, -1, 1], [2, 3, 99], [4, 5, 6], [7, -1, -1], [-7, 2 ** 31 - 1, 8]],
                     dtype=np.int32)
    c = stale_cache(rng, 9, heads, block, dim, "e4m3")
    c.append([0, 20], [20], table[1:2], *(bf16_values(rng, (20, heads, dim)) for _ in range(2)))
    dev = device_cache(c)
    rows = sum(new) + 6
    k, v = (bf16_values(rng, (rows, heads, dim)) for _ in range(2))
    q = bf16_values(rng, (rows, 4, dim))
    q_out = torch.full((rows, 4, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    at = starts(new)
    batch = device_batch(at, lens, table, rows=rows)
    mq.cache_append(dev, batch, device_bf16(k), device_bf16(v), q=device_bf16(q), q_out=q_out)
    c.append(at, lens, table, k, v)
    assert_cache_equal(dev, c)
    got = q_out.double().cpu().numpy()
    held = np.ones(rows, bool)
    held[sum(new):] = False
    held[at[3]:at[3] + 2] = False  # positions -2 and -1
    assert np.array_equal(got[held], q[held]) and np.all(got[~held] == 7)
    out = torch.full((rows, heads, dim), 5.0, device="cuda")
    out_v = out.clone()
    mq.cache_read(dev, batch, dtype=torch.float32, k_out=out, v_out=out_v)
    rk, rv = c.read(at, lens, table, rows)
    rk[sum(new):], rv[sum(new):] = 5.0, 5.0
    assert np.array_equal(out.cpu().numpy(), rk.astype(np.float32))
    assert np.array_equal(out_v.cpu().numpy(), rv.astype(np.float32))
    # attention over the same: pages that are not there hold no keys
    o = torch.full((rows, 4, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 4), 5.0, device="cuda")
    mq.cache_attend(dev, batch, device_bf16(q), out=o, lse=lse)
    ro, rl, info = c.attend(at, lens, table, q, dim ** -0.5)
    assert_attend(o, lse, ro, rl, info, dim, what="bad pages")
    assert torch.all(o[sum(new):] == 5) and torch.all(lse[sum(new):] == 5)
    assert np.isneginf(rl).any()


# ---------------------------------------------------------------- attend

def _attend_case(seed, lens, new, heads, group, block, dim, fmt, softcap=0.0, window=0, causal=True,
                 scale=None, wide=False, max_new=None, spread=1.0):
    rng = np.random.default_rng(seed)
    c, table = filled(rng, lens, heads, block, dim, fmt)
    at = starts(new)
    rows = int(at[-1])
    hq = heads * group
    q = bf16_values(rng, (rows, hq + (2 if wide else 0), dim), spread)
    dev = device_cache(c)
    batch = device_batch(at, lens, table, max_new=max_new)
    lse = torch.empty((rows, hq), dtype=torch.float32, device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    out = mq.cache_attend(dev, batch, device_bf16(q)[:, :hq], scale=scale, softcap=softcap,
                          window=window, causal=causal, lse=lse)
    ref, rl, info = c.attend(at, lens, table, q[:, :hq], scale, softcap, window, causal)
    assert_attend(out, lse, ref, rl, info, dim, softcap, f"{lens} {new} {dim} {fmt}")
    return dev, batch, q, out


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_attend_decode(block, dim, fmt):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 129, 300]
    new = [1, 1, 1, 1, 1, 1, 1, 1, 0, 1, 1, 1]
    _attend_case(block + dim, lens, new, 2, 3, block, dim, fmt)


@pytest.mark.parametrize("group,new,lens", [
    (1, [1, 1], [5, 700]),
    (4, [5, 3, 1], [400, 3, 77]),
    (8, [2, 0, 4], [130, 50, 4]),
    (7, [3, 1], [200, 1]),
    (20, [1, 2], [90, 333]),
    (4, [17, 40, 33], [17, 200, 100]),
    (1, [70, 200], [70, 450]),
    (2, [150, 1, 64, 128], [300, 280, 64, 129]),
    (4, [300], [301]),
])
@pytest.mark.parametrize("dim,fmt", [(64, "int8"), (128, "e4m3"), (128, "int8"), (256, "e4m3")])
def test_attend_tokens(group, new, lens, dim, fmt):
    _attend_case(group + dim, lens, new, 2, group, 32, dim, fmt)


@pytest.mark.parametrize("softcap,window,causal,new", [
    (30.0, 0, True, [1, 4, 20]), (0.0, 1, True, [1, 4, 20]), (0.0, 50, True, [1, 4, 20]),
    (0.0, 100000, True, [1, 4, 20]), (5.0, 64, True, [1, 4, 60]), (0.0, 0, False, [1, 4, 20]),
    (50.0, 0, False, [130, 4, 1]), (0.0, 33, True, [130, 64, 90]), (2.0, 0, True, [100, 3, 200]),
])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_masks_and_caps(softcap, window, causal, new, dim):
    _attend_case(3, [200, 131, 333], new, 1, 4, 64, dim, "e4m3" if dim == 128 else "int8",
                 softcap, window, causal, spread=4.0)


@pytest.mark.parametrize("new", [[1], [6], [90]])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attend_long_sequences_in_pieces(new, fmt):
    """Sequences cut into pieces, joined afterwards; strided queries."""
    dev, batch, q, out = _attend_case(8, [3111], new, 1, 2, 64, 64, fmt, wide=True, spread=3.0)
    assert mq.cache_attend_workspace_bytes(dev, batch, 2) > 0 or new[0] > 6


def test_attend_pieces_of_ragged_batches():
    """One long and several short sequences: some rows are written directly,
    some joined from pieces."""
    _attend_case(21, [2500, 3, 0, 700, 64], [1, 1, 0, 1, 1], 1, 4, 16, 128, "int8")
    _attend_case(22, [2500, 3, 0, 700, 64], [9, 2, 0, 5, 7], 1, 4, 16, 64, "e4m3", window=600)


@pytest.mark.parametrize("dim,fmt,group,softcap,window", [
    (64, "int8", 4, 0.0, 0), (128, "e4m3", 4, 0.0, 0), (256, "int8", 2, 30.0, 0),
    (128, "int8", 16, 0.0, 500), (128, "int8", 20, 0.0, 0)])
def test_attend_prompts_and_steps_of_one_batch(dim, fmt, group, softcap, window):
    """Chunks of prompts, drafted tokens, decode steps over short and long
    sequences and idle slots together: each goes its own way, some in pieces."""
    lens = [2500, 400, 1, 0, 1700, 65, 3000, 900]
    new = [1, 400, 1, 0, 3, 65, 130, 1]
    dev, batch, q, out = _attend_case(dim + group, lens, new, 2, group, 64, dim, fmt, softcap, window)
    again = mq.cache_attend(dev, batch, device_bf16(q), scale=dim ** -0.5, softcap=softcap,
                            window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_attend_prompts_among_many_sequences():
    """More sequences than a wave has lanes: prompts first, last and between,
    runs of idle slots, rows at the border of the two ways."""
    rng = np.random.default_rng(5)
    new = [1] * 150
    for i, n in ((0, 40), (63, 33), (64, 32), (65, 70), (100, 150), (149, 90)):
        new[i] = n
    for i in (1, 2, 62, 66, 67, 128, 140):
        new[i] = 0
    lens = [int(n + rng.integers(0, 200)) for n in new]
    _attend_case(6, lens, new, 2, 1, 32, 64, "int8")
    _attend_case(7, lens[:90], new[:90], 1, 4, 32, 128, "e4m3")


def test_attend_extreme_scores():
    """Scores of thousands and queries at the ends of bf16's range."""
    _attend_case(31, [150, 700], [2, 3], 2, 2, 32, 64, "int8", scale=3.0)
    _attend_case(32, [150, 90], [2, 70], 2, 2, 32, 128, "int8", scale=-2.0)
    rng = np.random.default_rng(33)
    c, table = filled(rng, [90, 90], 1, 32, 64, "int8")
    for size in (2.0 ** -126, 2.0 ** -100, 2.0 ** 60):
        for n in (2, 40):
            q = oracle.to_bf16(bf16_values(rng, (2 * n, 2, 64)) * size)
            s = float(np.float32(0.3 / size if size > 1e-38 and size < 1e30 else 1.0 / size))
            at = starts([n, n])
            lse = torch.empty((2 * n, 2), device="cuda")
            out = mq.cache_attend(device_cache(c), device_batch(at, [90, 90], table), device_bf16(q),
                                  scale=s, lse=lse)
            ref = c.attend(at, [90, 90], table, q, s)
            assert_attend(out, lse, *ref, 64, what=f"size {size}")


def test_attend_bad_queries_stay_alone():
    """A query of NaN or infinities leaves the other rows as they are."""
    rng = np.random.default_rng(34)
    c, table = filled(rng, [200], 1, 64, 64, "e4m3")
    dev = device_cache(c)
    for n in (4, 50):
        q = device_bf16(bf16_values(rng, (n, 4, 64)))
        batch = device_batch(starts([n]), [200], table)
        clean = mq.cache_attend(dev, batch, q)
        q2 = q.clone()
        q2[1, 2, 5] = float("nan")
        q2[n - 1, 0, 9] = float("inf")
        got = mq.cache_attend(dev, batch, q2)
        same = torch.ones((n, 4), dtype=torch.bool, device="cuda")
        same[1, 2], same[n - 1, 0] = False, False
        assert torch.equal(got[same], clean[same])
        assert not torch.isfinite(got[1, 2].float()).any()


def test_attend_zero_pages_and_uneven_scales():
    """Pages of zeros (scale 0) and of very different sizes in one sequence."""
    rng = np.random.default_rng(35)
    heads, block, dim = 1, 16, 64
    lens = [160]
    pages, table = make_table(rng, lens, block)
    for fmt in ("int8", "e4m3"):
        c = stale_cache(rng, pages, heads, block, dim, fmt)
        k, v = (bf16_values(rng, (160, 1, dim)) for _ in range(2))
        for i, f in enumerate([0, 1e-6, 1, 0, 1e4, 1e-20, 3, 0, 1e-3, 1]):
            v[16 * i:16 * i + 16] *= f
            k[16 * i:16 * i + 16] *= 0 if i in (0, 5) else 1
        c.append([0, 160], lens, table, oracle.to_bf16(k), oracle.to_bf16(v))
        for n in (1, 90):
            q = bf16_values(rng, (n, 2, dim))
            at = starts([n])
            lse = torch.empty((n, 2), device="cuda")
            out = mq.cache_attend(device_cache(c), device_batch(at, lens, table), device_bf16(q),
                                  lse=lse)
            assert_attend(out, lse, *c.attend(at, lens, table, q, dim ** -0.5), dim, what=fmt)


def test_attend_is_deterministic_and_plans_follow_their_tensors():
    rng = np.random.default_rng(36)
    c, table = filled(rng, [900, 40], 2, 64, 128, "int8")
    dev = device_cache(c)
    lens = device(np.array([900, 40], np.int32))
    batch = mq.KVBatch(device(starts([1, 1])), lens, device(table), rows=2, max_new=1)
    q = device_bf16(bf16_values(rng, (2, 8, 128)))
    plan = mq.CacheAttendPlan(dev, batch, q)
    a = plan().clone()
    assert torch.equal(plan(), a) and torch.equal(mq.cache_attend(dev, batch, q), a)
    lens.copy_(device(np.array([500, 7], np.int32)))
    ref = c.attend(starts([1, 1]), [500, 7], table, q.double().cpu().numpy(), 128 ** -0.5)
    assert_attend(plan(), None, *ref, 128, what="shorter")


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_then_steps(fmt):
    """A prompt in two chunks, then decode steps: rotation, cache and attention
    as they follow one another, each step against the oracle."""
    rng = np.random.default_rng(41)
    heads, group, block, dim, rot = 2, 3, 32, 64, 48
    total = 150
    pages, table = make_table(rng, [total, total], block)
    c = stale_cache(rng, pages, heads, block, dim, fmt)
    dev = device_cache(c)
    rope = _rope(rot, 1.1)
    have = [0, 0]
    for new in ([60, 31], [50, 70], [1, 1], [1, 1], [4, 1]):
        have = [a + b for a, b in zip(have, new)]
        at = starts(new)
        t = int(at[-1])
        x = rng.standard_normal((t, (group + 2) * heads, dim)).astype(np.float32)
        hq = group * heads
        xd = device(x)
        batch = device_batch(at, have, table)
        q = mq.cache_append(dev, batch, xd[:, hq:hq + heads], xd[:, hq + heads:], q=xd[:, :hq],
                            rope=rope)
        lse = torch.empty((t, hq), device="cuda")
        out = mq.cache_attend(dev, batch, q, lse=lse)
        pos = np.concatenate([np.arange(h - n, h) for h, n in zip(have, new)])
        turn = lambda y: oracle.to_bf16(oracle.rope_turn(y, pos, _freq(rot), 1.1))  # noqa: E731
        c.append(at, have, table, turn(x[:, hq:hq + heads]),
                 oracle.to_bf16(x[:, hq + heads:].astype(np.float64)))
        assert_cache_equal(dev, c)
        _same_bf16(q, turn(x[:, :hq]), "q")
        ref = c.attend(at, have, table, turn(x[:, :hq]), dim ** -0.5)
        assert_attend(out, lse, *ref, dim, what=str(new))


def test_captured_step_replays():
    """append and attend in one graph, replayed with longer sequences, with
    eager work between the replays."""
    rng = np.random.default_rng(42)
    heads, group, block, dim = 1, 4, 16, 64
    first = [700, 3]
    c, table = filled(rng, [740, 40], heads, block, dim, "int8")
    at0 = starts(first)
    c = stale_cache(rng, c.pages, heads, block, dim, "int8")
    c.append(at0, first, table, *(bf16_values(rng, (int(at0[-1]), heads, dim)) for _ in range(2)))
    dev = device_cache(c)
    lens = device(np.asarray(first, np.int32))
    x = torch.zeros((2, group + 2, dim), dtype=torch.bfloat16, device="cuda")
    batch = mq.KVBatch(device(starts([1, 1])), lens, device(table), rows=2, max_new=1)
    rope = _rope(64)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ap = mq.CacheAppendPlan(dev, batch, x[:, group:group + 1], x[:, group + 1:], q=x[:, :group],
                                rope=rope)
        q = ap.result
        at = mq.CacheAttendPlan(dev, batch, q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ap()
        at()
    for i in range(5):
        xv = bf16_values(rng, (2, group + 2, dim))
        x.copy_(device_bf16(xv))
        lens += 1
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        have = [n + i + 1 for n in first]
        pos = np.array(have) - 1
        turn = lambda y: oracle.to_bf16(oracle.rope_turn(y, pos, _freq(64)))  # noqa: E731
        c.append(starts([1, 1]), have, table, turn(xv[:, group:group + 1]), xv[:, group + 1:])
        assert_cache_equal(dev, c, f"replay {i}")
        ref = c.attend(starts([1, 1]), have, table, turn(xv[:, :group]), dim ** -0.5)
        assert_attend(at.result, None, *ref, dim, what=f"replay {i}")
        # the same step, eagerly, on the default stream
        batch2 = device_batch(starts([1, 1]), have, table)
        assert torch.equal(mq.cache_attend(dev, batch2, q), at.result)


def test_another_stream():
    rng = np.random.default_rng(43)
    c, table = filled(rng, [2000], 1, 64, 64, "int8")
    dev = device_cache(c)
    q = device_bf16(bf16_values(rng, (1, 4, 64)))
    batch = device_batch(starts([1]), [2000], table)
    want = mq.cache_attend(dev, batch, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [mq.cache_attend(dev, batch, q, stream=side) for _ in range(8)]
    side.synchronize()
    for g in got:
        assert torch.equal(g, want)


@pytest.mark.parametrize("block,dim", [(64, 128), (128, 256)])
def test_pool_beyond_four_gigabytes(block, dim):
    """Pages whose codes lie beyond 2^32 bytes: written, read and attended."""
    heads = 8
    per_page = heads * block * dim
    pages = (5 << 30) // per_page
    k = torch.zeros((pages, heads, block, dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros((pages, heads, dim, block), dtype=torch.uint8, device="cuda")
    s = torch.zeros((pages, heads), device="cuda")
    dev = mq.KVCache(k, v, s, s.clone(), "int8")
    rng = np.random.default_rng(44)
    n = block + 9
    table = np.array([[pages - 1, pages - 2]], dtype=np.int32)
    x = bf16_values(rng, (n, 2 * heads, dim))
    batch = device_batch(starts([n]), [n], table)
    xd = device_bf16(x)
    mq.cache_append(dev, batch, xd[:, :heads], xd[:, heads:])
    # the same tokens in a small pool
    c = oracle.Cache(np.zeros((2, heads, block, dim), np.uint8),
                     np.zeros((2, heads, dim, block), np.uint8),
                     np.zeros((2, heads), np.float32), np.zeros((2, heads), np.float32), "int8")
    low = np.array([[1, 0]], dtype=np.int32)
    c.append(starts([n]), [n], low, x[:, :heads], x[:, heads:])
    assert np.array_equal(k[-2:].cpu().numpy(), c.k) and np.array_equal(v[-2:].cpu().numpy(), c.v)
    assert int(k[:-2].count_nonzero()) == 0 and int(v[:-2].count_nonzero()) == 0
    rk, _ = mq.cache_read(dev, batch, dtype=torch.float32)
    assert np.array_equal(rk.cpu().numpy(), c.read(starts([n]), [n], low, n)[0].astype(np.float32))
    last = device_batch(starts([1]), [n], table)
    q = bf16_values(rng, (1, heads, dim))
    out = mq.cache_attend(dev, last, device_bf16(q))
    assert_attend(out, None, *c.attend(starts([1]), [n], low, q, dim ** -0.5), dim, what="far")


# ---------------------------------------------------------------- refusals on the GPU

def test_python_refusals():
    rng = np.random.default_rng(45)
    c, table = filled(rng, [20], 2, 16, 64, "int8")
    dev = device_cache(c)
    batch = device_batch(starts([2]), [20], table)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    rope = _rope(64)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mq.rope(x.half(), rope, pos)
    with pytest.raises(TypeError):
        mq.rope(x, rope, pos.long())
    with pytest.raises(ValueError):
        mq.rope(x, rope, pos[:1])
    with pytest.raises(ValueError):
        mq.rope(x.transpose(1, 2), rope, pos)
    with pytest.raises(ValueError):
        mq.rope(x[:1].expand(2, 2, 64), rope, pos)
    with pytest.raises(ValueError):
        mq.rope(x.cpu(), rope, pos)
    with pytest.raises(mq.MQError):
        mq.rope(x, _rope(128), pos)
    with pytest.raises(ValueError):
        mq.cache_append(dev, batch, x[:1], x)
    with pytest.raises(ValueError):
        mq.cache_append(dev, batch, x, x.float())
    with pytest.raises(TypeError):
        mq.cache_append(dev, batch, x, x, q=x.float())
    with pytest.raises(ValueError):
        mq.cache_append(dev, batch, x, x, q_out=x)
    with pytest.raises(ValueError):
        mq.cache_attend(dev, batch, x[:, :, :32])
    with pytest.raises(TypeError):
        mq.cache_attend(dev, batch, x.float())
    with pytest.raises(mq.MQError):
        mq.cache_attend(dev, batch, torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mq.MQError):
        mq.cache_attend(dev, batch, x, window=4, causal=False)
    with pytest.raises(TypeError):
        mq.cache_read(dev, batch, dtype=torch.float16)
    with pytest.raises(ValueError):
        mq.cache_attend(dev, batch, x, lse=torch.zeros((2, 3), device="cuda"))
