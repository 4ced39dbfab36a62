"""The Mix'n'Match stack with attention (mq_mixnmatch_attend): every layer run
alone with each step checked from the GPU's own inputs to it (rotation and
codes bit for bit, attention and products within their bounds), the whole
stack against its layers, decode steps in a captured graph."""

import numpy as np
import pytest
import torch

import nested_int_matmul_amd as mq
import oracle
from attention_helpers import (assert_attend, assert_cache_equal, device, device_batch, device_cache,
                               make_table, stale_cache, starts)
from gpu_helpers import compare_linear, dev, x_device

pytestmark = pytest.mark.gpu

DIM, HEADS, GROUP, F = 64, 2, 3, 512
H = DIM * HEADS * GROUP
ROT = 32
SHAPES = {"q": (H, H), "k": (HEADS * DIM, H), "v": (HEADS * DIM, H), "o": (H, H), "up": (F, H),
          "gate": (F, H), "down": (H, F)}


def _layers(rs, seed):
    rng = np.random.default_rng(seed)
    host, devl = [], []
    for r in rs:
        hl, dl = {"r": r}, {"r": r}
        for name, (n, k) in SHAPES.items():
            w = rng.standard_normal((n, k)).astype(np.float32) * np.float32(0.05)
            q, a, z = oracle.quantize_minmax(w, k)
            hl[name] = {"q": q, "alpha": a, "zero": z, "group": k}
            dl[name] = {"packed": mq.pack(torch.from_numpy(q).to(dev()), r),
                        "alpha": torch.from_numpy(a).to(dev()),
                        "zero": torch.from_numpy(z).to(dev()), "N": n, "K": k, "group": k}
        host.append(hl)
        devl.append(dl)
    return host, devl


def _x(rng, m):
    return oracle.bf16_bits_from_float(rng.standard_normal((m, H)))


def _freq():
    return 10000.0 ** (-np.arange(0, ROT, 2) / ROT)


@pytest.mark.parametrize("fmt,new,rs,windows,softcap", [
    ("int8", [1, 1, 0, 1], [8, 4, 2], None, 0.0),
    ("e4m3", [5, 3], [4, 4], [0, 9], 0.0),
    ("int8", [8], [8, 3], None, 20.0),
    ("e4m3", [1], [6], [4], 0.0),
])
def test_layers_step_by_step(fmt, new, rs, windows, softcap):
    rng = np.random.default_rng(len(new) * 7 + len(rs))
    host, devl = _layers(rs, 3)
    m = sum(new)
    first = [20, 3, 0, 33][:len(new)]
    lens = [a + b for a, b in zip(first, new)]
    block = 16
    pages, table = make_table(rng, lens, block)
    refs = [stale_cache(rng, pages, HEADS, block, DIM, fmt) for _ in rs]
    for c in refs:
        at0 = starts(first)
        c.append(at0, first, table, *(oracle.to_bf16(rng.standard_normal((int(at0[-1]), HEADS, DIM)))
                                      for _ in range(2)))
    caches = [device_cache(c) for c in refs]
    whole = [device_cache(c) for c in refs]
    rope = mq.Rope(device(_freq()), 1.0)
    at = starts(new)
    batch = device_batch(at, lens, table)
    pos = np.concatenate([np.arange(a, b) for a, b in zip(first, lens)])
    xb = _x(rng, m)
    h = x_device(xb).view(torch.bfloat16).float().reshape(m, H)
    for i, r in enumerate(rs):
        one = mq.make_layers(devl[i:i + 1])
        attn = mq.StackAttention(caches[i:i + 1], batch, HEADS * GROUP, rope=rope, softcap=softcap,
                                 windows=windows[i:i + 1] if windows else None)
        ws = torch.empty(mq.mixnmatch_attend_workspace_bytes(one, attn, m), dtype=torch.uint8,
                         device=dev())
        before = h.clone()
        assert mq.mixnmatch_attend(one, attn, h=h, workspace=ws) is h
        off = mq.mixnmatch_workspace_offsets(one, m)
        base = mq.mixnmatch_workspace_bytes(one, m)

        def f32(j, n):
            return ws[off[j]:off[j] + m * n * 4].view(torch.float32).reshape(m, n)

        q, k, v = (f32(j, n).double().cpu().numpy().reshape(m, -1, DIM)
                   for j, n in ((1, H), (2, HEADS * DIM), (3, HEADS * DIM)))
        turn = lambda y: oracle.to_bf16(oracle.rope_turn(y, pos, _freq()))  # noqa: E731
        refs[i].append(at, lens, table, turn(k), oracle.to_bf16(v))
        assert_cache_equal(caches[i], refs[i], f"layer {i}")
        qr = ws[off[8]:off[8] + m * H * 2].view(torch.bfloat16).reshape(m, HEADS * GROUP, DIM)
        assert np.array_equal(qr.double().cpu().numpy(), turn(q))
        out = ws[base:base + m * H * 2].view(torch.bfloat16).reshape(m, HEADS * GROUP, DIM)
        ref = refs[i].attend(at, lens, table, turn(q), DIM ** -0.5, softcap,
                             windows[i] if windows else 0)
        assert_attend(out, None, *ref, DIM, softcap, f"layer {i}")
        o, d = f32(6, H), f32(7, H)
        p = host[i]["o"]
        ob = out.reshape(m, H).contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        compare_linear(o, ob, p["q"], p["alpha"], p["zero"], p["group"], r, f"layer {i} o")
        assert torch.equal(h, before + o + d)
    # all layers in one call, from the bf16 input: the same numbers
    attn = mq.StackAttention(whole, batch, HEADS * GROUP, rope=rope, softcap=softcap,
                             windows=windows)
    got = mq.mixnmatch_attend(mq.make_layers(devl), attn, x=x_device(xb).reshape(m, H))
    assert torch.equal(got, h)
    for a, b in zip(whole, caches):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_decode_steps_in_a_graph():
    rng = np.random.default_rng(5)
    _, devl = _layers([8, 4], 4)
    block, first, steps = 32, [30, 200], 4
    lens0 = [n + steps for n in first]
    pages, table = make_table(rng, lens0, block)
    refs = [stale_cache(rng, pages, HEADS, block, DIM, "int8") for _ in range(2)]
    for c in refs:
        at0 = starts(first)
        c.append(at0, first, table, *(oracle.to_bf16(rng.standard_normal((int(at0[-1]), HEADS, DIM)))
                                      for _ in range(2)))
    eager, graphed = ([device_cache(c) for c in refs] for _ in range(2))
    rope = mq.Rope(device(_freq()), 1.0)
    lens = device(np.asarray(first, np.int32))
    batch = mq.KVBatch(device(starts([1, 1])), lens, device(table), rows=2, max_new=1)
    arr = mq.make_layers(devl)
    x = torch.zeros((2, H), dtype=torch.bfloat16, device="cuda")
    a_graph = mq.StackAttention(graphed, batch, HEADS * GROUP, rope=rope)
    a_eager = mq.StackAttention(eager, batch, HEADS * GROUP, rope=rope)
    out = torch.empty((2, H), device="cuda")
    ws = torch.empty(mq.mixnmatch_attend_workspace_bytes(arr, a_graph, 2), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.mixnmatch_attend(arr, a_graph, x=x, h=out, workspace=ws)
    for i in range(steps):
        x.copy_(torch.from_numpy(rng.standard_normal((2, H)).astype(np.float32)))
        lens += 1
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = mq.mixnmatch_attend(arr, a_eager, x=x)
        assert torch.equal(out, want), f"step {i}"
        for a, b in zip(graphed, eager):
            assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
            assert torch.equal(a.k_scale.isnan(), b.k_scale.isnan())


def test_refusals():
    rng = np.random.default_rng(6)
    _, devl = _layers([8], 4)
    pages, table = make_table(rng, [9], 16)
    cache = device_cache(stale_cache(rng, pages, HEADS, 16, DIM, "int8"))
    batch = device_batch(starts([2]), [9], table)
    arr = mq.make_layers(devl)
    x = torch.zeros((2, H), dtype=torch.bfloat16, device="cuda")
    good = mq.StackAttention([cache], batch, HEADS * GROUP)
    for bad in (mq.StackAttention([cache], batch, HEADS),
                mq.StackAttention([cache], batch, HEADS * GROUP, windows=[-1]),
                mq.StackAttention([cache], batch, HEADS * GROUP, scale=float("nan")),
                mq.StackAttention([device_cache(stale_cache(rng, 2, 2 * HEADS, 16, DIM, "int8"))],
                                  batch, 2 * HEADS)):
        assert mq.mixnmatch_attend_workspace_bytes(arr, bad, 2) == 0
        with pytest.raises(mq.MQError):
            mq.mixnmatch_attend(arr, bad, x=x)
    with pytest.raises(ValueError):
        mq.StackAttention([], batch, HEADS)
    with pytest.raises(ValueError):
        mq.StackAttention([cache], batch, HEADS * GROUP, windows=[0, 0])
    with pytest.raises(ValueError):
        mq.mixnmatch_attend(arr, good, x=x[:1])
    with pytest.raises(ValueError):
        mq.mixnmatch_attend(arr, good)
    with pytest.raises(mq.MQError):
        mq.mixnmatch_attend(arr, good, x=x, workspace=torch.empty(256, dtype=torch.uint8,
                                                                   device="cuda"))
