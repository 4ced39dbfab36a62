"""Builds caches, batches and inputs of the attention tests on the CPU (numpy)
and puts the same on the GPU."""

from __future__ import annotations

import numpy as np
import torch

import nested_int_matmul_amd as mq
import oracle


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def bf16_values(rng, shape, spread=4.0):
    """bf16 numbers as float64, a few channels larger than the rest."""
    x = rng.standard_normal(shape)
    x[..., ::16] *= spread
    return oracle.to_bf16(x)


def make_table(rng, lens, block, spare=2):
    """Shuffled pages for sequences of `lens` tokens: (pages, int32 table).
    Entries behind a sequence's last page are -1."""
    per = [-(-max(0, int(x)) // block) for x in lens]
    pages = sum(per) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(1, max(per))), -1, dtype=np.int32)
    at = 0
    for s, p in enumerate(per):
        table[s, :p] = order[at:at + p]
        at += p
    return pages, table


def stale_cache(rng, pages, heads, block, dim, fmt):
    """A cache full of earlier use: any byte (e4m3's NaN patterns too), scales
    that are no numbers.  Nothing of it may be seen."""
    k = rng.integers(0, 256, (pages, heads, block, dim), dtype=np.uint8)
    v = rng.integers(0, 256, (pages, heads, dim, block), dtype=np.uint8)
    s = np.full((pages, heads), np.nan, dtype=np.float32)
    return oracle.Cache(k, v, s, s.copy(), fmt)


def device(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")


def device_bf16(x):
    return device(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def device_cache(c):
    return mq.KVCache(device(c.k), device(c.v), device(c.ks), device(c.vs), c.fmt)


def device_batch(q_start, kv_len, table, rows=None, max_new=None):
    n = np.diff(q_start)
    return mq.KVBatch(device(np.asarray(q_start, np.int32)), device(np.asarray(kv_len, np.int32)),
                      device(np.asarray(table, np.int32)),
                      rows=int(q_start[-1]) if rows is None else rows,
                      max_new=max(1, int(n.max())) if max_new is None else max_new)


def filled(rng, lens, heads, block, dim, fmt):
    """A stale cache into which the oracle wrote `lens` tokens; its table."""
    pages, table = make_table(rng, lens, block)
    c = stale_cache(rng, pages, heads, block, dim, fmt)
    at = starts(lens)
    k, v = (bf16_values(rng, (int(at[-1]), heads, dim)) for _ in range(2))
    c.append(at, np.asarray(lens), table, k, v)
    return c, table


def assert_cache_equal(dev, ref, what=""):
    """Every byte and scale of the whole pool."""
    assert np.array_equal(dev.k.cpu().numpy(), ref.k), f"{what}: k codes"
    assert np.array_equal(dev.v.cpu().numpy(), ref.v), f"{what}: v codes"
    for got, want, name in ((dev.k_scale, ref.ks, "k"), (dev.v_scale, ref.vs, "v")):
        assert np.array_equal(got.cpu().numpy().view(np.int32), want.view(np.int32)), \
            f"{what}: {name} scales"


def attend_bounds(out, lse, info, dim, softcap=0.0):
    """Largest deviations of the fp32 arithmetic (entry by entry) from the
    float64 result.  u = 2^-24 is half a step of fp32.

    A score is a sum of `dim` exact products in fp32 (error at most dim u times
    the sum of their magnitudes, `size`), a product with the scales (3 u) and,
    with a cap, a tanh whose error is below 2^-20 of it.  exp2 turns a score's
    error e (it and the reference's, 2 u |t| each) into a relative one: e on
    each probability and, through the sum, on the normalization.  The
    probability is rounded to fp16 (half a step 2^-11) in units of the row's
    reference, below 2^-14 with an absolute error 2^-25 of v's largest; the
    scales' unit adds 4 u.  The result is rounded to bf16: 2^-8 of it."""
    u = 2.0 ** -24
    size = info["size"]
    e = (dim + 8) * u * size + 8 * u * (np.abs(np.where(np.isfinite(lse), lse, 0)) + size)
    if softcap:
        e = e + 2.0 ** -20 * np.minimum(size, softcap)
    e = e + 2.0 ** -21  # exp2 and log2 of the unit, sums of probabilities
    per = (2.0 ** -11 + 3 * e)[..., None] * info["mass"]
    tiny = (2.0 ** -25 * info["seen"] * info["vmax"])[..., None]
    o = np.where(np.isfinite(out), np.abs(out), 0)
    return (per + tiny) * (1 + 2.0 ** -7) + 2.0 ** -8 * o + 1e-37, 2 * e


def assert_attend(got, got_lse, out, lse, info, dim, softcap=0.0, what=""):
    b_out, b_lse = attend_bounds(out, lse, info, dim, softcap)
    g = got.double().cpu().numpy()
    live = ~np.isnan(lse)  # rows of a sequence
    assert np.all(np.isfinite(g[live])), f"{what}: non-finite output"
    err = np.abs(g - out)[live]
    worst = float((err / b_out[live]).max()) if err.size else 0.0
    line = f"  {what}: output error / bound {worst:.3f}"
    assert worst <= 1.0, line
    if got_lse is not None:
        gl = got_lse.double().cpu().numpy()[live]
        rl = lse[live]
        none = np.isneginf(rl)
        assert np.array_equal(none, np.isneginf(gl)), f"{what}: rows without keys"
        assert np.all(g[live][none] == 0), f"{what}: rows without keys"
        le = np.abs(gl - rl)[~none] / b_lse[live][~none]
        worst = float(le.max()) if le.size else 0.0
        line += f", lse {worst:.3f}"
        assert worst <= 1.0, line
    print(line, flush=True)
