"""Measured cases of the serving operators around attention: rotary positions,
the 8-bit key/value cache (written and read back) and attention over it.

Every case is one operator call at one set of sizes.  `run` computes it in
plain torch, or, with `own` set, through nested_int_matmul_amd.  Head layouts
are those of the models whose layers the framework serves: 32 query and 8
key/value heads of 128, and 16 query and 8 key/value heads of 256; the other
layouts are generic.

The cache: pages of `block` tokens; k codes [pages, heads, block, dim], v codes
[pages, heads, dim, block], one fp32 scale per page and head for each; int8
(scale amax / 127) or e4m3 (amax / 448).  A sequence's pages are listed in its
row of the page table; its last tokens are the call's rows.
"""

import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "e4m3": 448.0}
MIN_SCALE = 2.0 ** -100


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 8 sequences: the queries of one layer, as the fp32 product leaves them
        dict(name="rope_decode", op="rope", rows=8, heads=32, dim=128, rot=128, interleaved=False,
             x="fp32", scaling="none", fused=False, far=32768),
        # a whole prompt's queries in bf16, frequencies scaled for a context four times the trained one
        dict(name="rope_prompt", op="rope", rows=8192, heads=32, dim=128, rot=128,
             interleaved=False, x="bf16", scaling="yarn", fused=False, far=131072),
        # a ragged chunk, a quarter of each head rotated, queries inside the fused q|k|v rows
        dict(name="rope_part", op="rope", rows=1531, heads=16, dim=256, rot=64, interleaved=True,
             x="fp32", scaling="linear", fused=True, far=65536),
        # one decode step of 32 sequences: k and v of one token each into the cache, k and q rotated
        dict(name="append_decode", op="append", seqs=32, new=1, ctx=1000, heads=8, group=4, dim=128,
             rot=128, block=64, fmt="e4m3", x="fp32", rotate_q=True),
        # one prompt of 8192 tokens written to an empty cache
        dict(name="append_prompt", op="append", seqs=1, new=8192, ctx=8192, heads=8, group=2,
             dim=256, rot=256, block=128, fmt="e4m3", x="bf16", rotate_q=True),
        # chunks of several sequences that begin inside a page, then the sequences read back
        dict(name="append_chunks_read", op="append", seqs=6, new=700, ctx=1500, heads=8, group=4,
             dim=128, rot=64, block=32, fmt="int8", x="bf16", rotate_q=False),
        # long sequences brought back to bf16, as a prefix is moved or re-used elsewhere
        dict(name="read_long", op="read", seqs=4, ctx=16384, heads=8, dim=128, block=64,
             fmt="e4m3", out="bf16"),
        # a few short sequences read back in fp32
        dict(name="read_short", op="read", seqs=3, ctx=333, heads=4, dim=64, block=16,
             fmt="int8", out="fp32"),
        # one user, one token, a short context: latency
        dict(name="attend_short", op="attend", seqs=1, new=1, ctx=700, heads=8, group=4, dim=128,
             block=64, fmt="int8", window=0, softcap=0.0),
        # a decode batch of sequences of very different lengths, an idle slot among them
        dict(name="attend_batch", op="attend", seqs=32, new=1, ctx=16384, heads=8, group=4, dim=128,
             block=64, fmt="int8", window=0, softcap=0.0),
        # five drafted tokens a sequence checked at once; heads of 256, a local layer of 4096
        # tokens, scores capped at 50
        dict(name="attend_drafts", op="attend", seqs=8, new=5, ctx=8000, heads=8, group=2, dim=256,
             block=32, fmt="e4m3", window=4096, softcap=50.0),
        # a chunk of a long prompt beside shorter ones: bound by the products
        dict(name="attend_prompt", op="attend", seqs=2, new=2048, ctx=8192, heads=8, group=4,
             dim=128, block=64, fmt="int8", window=0, softcap=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8])
    block = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["int8", "e4m3"])
    if op == "rope":
        heads = rng.choice([1, 4, 7, 16, 32])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 24])
        return dict(op=op, rows=_log(rng, 1, 8192 * 4096 // (heads * dim) // 4), heads=heads, dim=dim,
                    rot=rot, interleaved=rng.random() < 0.5, x=rng.choice(["fp32", "bf16"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), fused=rng.random() < 0.5,
                    far=rng.choice([2048, 131072]))
    if op == "append":
        seqs = _log(rng, 1, 48)
        new = _log(rng, 1, max(1, 8192 // seqs))
        return dict(op=op, seqs=seqs, new=new, ctx=new + _log(rng, 1, 1000), heads=heads,
                    group=rng.choice([1, 2, 4, 7]), dim=dim, rot=rng.choice([0, dim, dim // 2, 24]),
                    block=block, fmt=fmt, x=rng.choice(["fp32", "bf16"]),
                    rotate_q=rng.random() < 0.5)
    if op == "read":
        seqs = _log(rng, 1, 16)
        return dict(op=op, seqs=seqs, ctx=_log(rng, 1, 32768 // seqs), heads=heads, dim=dim,
                    block=block, fmt=fmt, out=rng.choice(["fp32", "bf16"]))
    new = rng.choice([1, 1, 2, 4, 5, 8, 0])
    group = rng.choice([1, 2, 4, 5, 8])
    if new == 0:  # a chunk of prompts
        seqs, group = rng.choice([1, 2]), rng.choice([1, 2, 4])
        new = _log(rng, 16, 1000)
        ctx = new + _log(rng, 1, 4096)
    else:
        seqs = _log(rng, 1, 48)
        ctx = new + _log(rng, 1, min(131072, 262144 // (seqs * max(1, heads * dim // 512))))
    return dict(op=op, seqs=seqs, new=new, ctx=ctx, heads=heads, group=group, dim=dim, block=block,
                fmt=fmt, window=rng.choice([0, 0, 0, 100, 4096]), softcap=rng.choice([0.0, 0.0, 30.0]))


def _lengths(case):
    """New tokens and cached tokens (with the new ones) of each sequence.  The first is the
    longest; one slot in eight of a larger batch is idle, and one sequence has just begun."""
    rng = random.Random("%d %d %d" % (case["seqs"], case.get("new", 0), case["ctx"]))
    n, length = [], []
    for s in range(case["seqs"]):
        whole = "new" not in case
        top = case["ctx"] if whole else case["new"]
        if s == 0:
            a, b = top, case["ctx"]
        elif s % 8 == 5:
            a, b = 0, 0
        elif s % 8 == 3:
            a = rng.randint(1, top)
            b = a
        else:
            a = rng.randint(max(1, top // 3), top)
            b = a if whole else rng.randint(a + (case["ctx"] - top) // 8, a + case["ctx"] - top)
        n.append(a)
        length.append(a if whole else b)
    return n, length


def _seen(case):
    """(visible (query, key) pairs, distinct keys) over all sequences."""
    pairs = keys = 0
    w = case["window"]
    for n, length in zip(*_lengths(case)):
        for_all = [min(length - n + i + 1, w) if w else length - n + i + 1 for i in range(n)]
        pairs += sum(for_all)
        keys += min(length, w + n - 1) if w and n else (length if n else 0)
    return pairs, keys


def work(case):
    op = case["op"]
    size = 4 if case.get("x", case.get("out")) == "fp32" else 2
    if op == "rope":
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": n * (size + 2) + case["rows"] * 4, "flops": 3 * n}
    h, d = case["heads"], case["dim"]
    n, length = _lengths(case)
    if op == "append":
        rows = sum(n)
        kv, q = 2 * rows * h * d, rows * h * case["group"] * d if case["rotate_q"] else 0
        got = {"bytes": kv * (size + 1) + q * (size + 2), "flops": 4 * (kv + q)}
        if case["fmt"] == "int8":  # read back
            got["bytes"] += 2 * sum(length) * h * d * 5
        return got
    if op == "read":
        kv = 2 * sum(n) * h * d
        return {"bytes": kv * (1 + size), "flops": kv}
    pairs, keys = _seen(case)
    hq = h * case["group"]
    return {"bytes": 2 * keys * h * d + sum(n) * hq * (d * 4 + 4), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the inputs

def _frequencies(case):
    """Radians a position for each pair (float64), and the factor of the rotated values."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    kind, factor, trained = case.get("scaling", "none"), 4.0, 32768
    if kind == "linear":
        return f / factor, 1.0
    if kind == "yarn":  # slow pairs interpolated, fast ones kept, a ramp between 1 and 32 turns
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _values(g, shape, dtype, spread=0):
    """Normal values; with `spread`, every 16th entry of the last axis is larger by that factor."""
    t = torch.randn(shape, generator=g, device=DEV)
    if spread:
        t[..., ::16] *= spread
    return t.to(dtype)


def _codes(t, fmt, axes):
    """Codes and scales of whole pages of values."""
    s = t.abs().amax(dim=axes) / QMAX[fmt]
    q = t / s[..., None, None]
    q = q.to(torch.float8_e4m3fn) if fmt == "e4m3" else q.round().to(torch.int8)
    return q.view(torch.uint8), s


def _cache(case, g, length):
    """A pool of shuffled pages that holds `length` tokens of each sequence, and its page table."""
    b, h, d = case["block"], case["heads"], case["dim"]
    per = [-(-x // b) for x in length]
    pages, wide = sum(per) + 3, max(1, max(per))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at, rows = 0, []
    for p in per:
        rows.append(torch.cat([order[at:at + p], order.new_zeros(wide - p)]))
        at += p
    k, ks = _codes(_values(g, (pages, h, b, d), torch.float32, 4), case["fmt"], (2, 3))
    v, vs = _codes(_values(g, (pages, h, d, b), torch.float32), case["fmt"], (2, 3))
    return dict(k=k, v=v, ks=ks, vs=vs, table=torch.stack(rows))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(n):
    got = [0]
    for x in n:
        got.append(got[-1] + x)
    return got


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    st = dict(case=case)
    op, d = case["op"], case["dim"]
    xt = torch.float32 if case.get("x") == "fp32" else torch.bfloat16
    if case.get("rot"):
        f, st["factor"] = _frequencies(case)
        st["freq"] = f.to(DEV)
    if op == "rope":
        t, h = case["rows"], case["heads"]
        x = _values(g, (t, 2 * h, d) if case["fused"] else (t, h, d), xt)
        st["x"] = x[:, :h]
        if t > 64:  # a chunk of one prompt
            begin = int(torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=DEV))
            st["pos"] = torch.arange(begin, begin + t, device=DEV, dtype=torch.int32)
        else:  # tokens of different sequences
            st["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV).to(torch.int32)
    else:
        h = case["heads"]
        n, length = _lengths(case)
        st["rows"], st["most"] = sum(n), max(n)
        st["start"], st["len"] = _ints(_starts(n)), _ints(length)
        st.update(_cache(case, g, length))
        if op == "append":
            hq = h * case["group"]
            x = _values(g, (st["rows"], hq + 2 * h, d), xt, 3)
            st["q"] = x[:, :hq] if case["rotate_q"] else None
            st["new_k"], st["new_v"] = x[:, hq:hq + h], x[:, hq + h:]
            st["start_all"], st["rows_all"] = _ints(_starts(length)), sum(length)
        if op == "attend":
            st["q"] = _values(g, (st["rows"], h * case["group"], d), torch.bfloat16)
            st["scale"] = d ** -0.5
    if own:
        _own_prepare(st)
    return st


# ------------------------------------------------------------------ the framework's calls

def _own_prepare(st):
    """The handles that a serving loop keeps: the cache, the batch's description and, for
    decode steps, the prepared call."""
    import nested_int_matmul_amd as mq

    case, op = st["case"], st["case"]["op"]
    st["mq"] = mq
    st["rope"] = mq.Rope(st["freq"], interleaved=case.get("interleaved", False),
                         factor=st["factor"]) if case.get("rot") else None
    st["call"] = None
    if op == "rope":
        if case["rows"] <= 64:
            out = torch.empty(tuple(st["x"].shape), dtype=torch.bfloat16, device=DEV)
            st["call"] = mq.RopePlan(st["x"], st["rope"], st["pos"], out=out)
        return
    st["cache"] = mq.KVCache(st["k"], st["v"], st["ks"], st["vs"], case["fmt"])
    st["batch"] = mq.KVBatch(st["start"], st["len"], st["table"], rows=st["rows"],
                             max_new=st["most"])
    if op == "append":
        st["batch_all"] = mq.KVBatch(st["start_all"], st["len"], st["table"],
                                     rows=st["rows_all"], max_new=case["ctx"])
        if st["rows"] <= 64 and case["fmt"] == "e4m3":
            st["call"] = mq.CacheAppendPlan(st["cache"], st["batch"], st["new_k"], st["new_v"],
                                            q=st["q"], rope=st["rope"])
    if op == "attend" and st["rows"] <= 64:
        out = torch.empty_like(st["q"])
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
        st["call"] = mq.CacheAttendPlan(st["cache"], st["batch"], st["q"], scale=st["scale"],
                                        softcap=case["softcap"], window=case["window"], out=out,
                                        lse=lse)


def _own_run(st):
    mq, case, op = st["mq"], st["case"], st["case"]["op"]
    if op == "rope":
        if st["call"] is not None:
            return st["call"]()
        return mq.rope(st["x"], st["rope"], st["pos"])
    if op == "append":
        if st["call"] is not None:
            q = st["call"]()
        else:
            q = mq.cache_append(st["cache"], st["batch"], st["new_k"], st["new_v"], q=st["q"],
                                rope=st["rope"])
        if case["fmt"] == "e4m3":
            return _pool(st, q)
        k, v = mq.cache_read(st["cache"], st["batch_all"], dtype=torch.float32)
        return dict(q=q, k=k, v=v, ks=st["ks"], vs=st["vs"])
    if op == "read":
        return mq.cache_read(st["cache"], st["batch"],
                             dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    if st["call"] is not None:
        return st["call"]()
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    out = mq.cache_attend(st["cache"], st["batch"], st["q"], scale=st["scale"],
                          softcap=case["softcap"], window=case["window"], lse=lse)
    return out, lse


# ------------------------------------------------------------------ the plain forms

def _pool(st, q):
    """The whole updated cache: e4m3 codes as the numbers they are, and their scales."""
    return dict(q=q, k=st["k"].view(torch.float8_e4m3fn), v=st["v"].view(torch.float8_e4m3fn),
                ks=st["ks"], vs=st["vs"])


def _rotate(x, pos, freq, factor, interleaved):
    """Rotary positions in 64 bits (angles of far positions; and the cache's codes are next to
    borders), rounded once to fp32 and from there to bf16."""
    a = pos.double()[:, None] * freq
    c, s = (torch.cos(a) * factor)[:, None], (torch.sin(a) * factor)[:, None]
    x = x.double()
    rot = 2 * freq.numel()
    if interleaved:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1).float().to(torch.bfloat16)


def _round_codes(x, fmt):
    """Float64 quotients to the nearest code, ties to even, as numbers."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2((torch.frexp(x).exponent - 1).clamp(min=-6).double() - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _as_bytes(x, fmt):
    return (x.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else x.to(torch.int8)).view(torch.uint8)


def _as_numbers(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _write(codes, scales, x, page, slot, part, used, fmt, tokens_last):
    """New rows x [T, H, D] (bf16) into pages `page`, places `slot`.  `part`: pages that already
    hold `used` earlier tokens."""
    amax = torch.zeros_like(scales)
    amax.index_reduce_(0, page, x.abs().amax(-1).float(), "amax")
    fresh = amax / QMAX[fmt]
    fresh = torch.where(fresh < MIN_SCALE, torch.zeros_like(fresh), fresh)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=scales.device)
    touched[page] = True
    old = torch.zeros_like(scales)
    old[part] = scales[part]
    now = torch.where(touched[:, None], torch.maximum(old, fresh), scales)
    # earlier codes of the pages whose scale grew
    c = _as_numbers(codes[part], fmt).double()
    if tokens_last:
        c = c.transpose(2, 3)
    ratio_new = torch.where(now[part] > 0, now[part], torch.ones_like(now[part])).double()
    again = _round_codes(c * old[part].double()[..., None, None] / ratio_new[..., None, None], fmt)
    earlier = torch.arange(c.shape[2], device=c.device)[None, None, :, None] < used[:, None, None, None]
    grew = (now[part] > old[part])[..., None, None]
    c = torch.where(earlier & grew, again, c)
    if tokens_last:
        c = c.transpose(2, 3)
    codes[part] = _as_bytes(c, fmt)
    # the new codes
    s = now[page]
    y = x.double() / torch.where(s > 0, s, torch.full_like(s, math.inf)).double()[..., None]
    y = _as_bytes(_round_codes(y, fmt), fmt)
    if tokens_last:
        codes[page, :, :, slot] = y
    else:
        codes[page, :, slot] = y
    scales.copy_(now)


def _places(start, length, rows, block, table):
    """Position, page and place in the page of every row."""
    r = torch.arange(rows, device=start.device)
    s = torch.searchsorted(start[1:].long(), r, right=True)
    pos = length.long()[s] - start.long()[s + 1] + r
    return pos, table.long()[s, pos // block], pos % block


def _gather(st, dtype):
    pos, page, slot = _places(st["start"], st["len"], st["rows"], st["case"]["block"], st["table"])
    return _gather_at(st, page, slot, dtype)


def _gather_at(st, page, slot, dtype):
    fmt = st["case"]["fmt"]
    k = _as_numbers(st["k"][page, :, slot], fmt) * st["ks"][page][..., None]
    v = _as_numbers(st["v"][page, :, :, slot], fmt) * st["vs"][page][..., None]
    return k.to(dtype), v.to(dtype)


def _plain_append(st):
    case = st["case"]
    fmt, b = case["fmt"], case["block"]
    pos, page, slot = _places(st["start"], st["len"], st["rows"], b, st["table"])
    k, v, q = st["new_k"].to(torch.bfloat16), st["new_v"].to(torch.bfloat16), st["q"]
    if case["rot"]:
        k = _rotate(st["new_k"], pos, st["freq"], st["factor"], False)
    if q is not None:
        q = _rotate(q, pos, st["freq"], st["factor"], False) if case["rot"] else q.to(torch.bfloat16)
    n = (st["start"][1:] - st["start"][:-1]).long()
    begin = st["len"].long() - n
    has = (n > 0) & (begin % b > 0)
    part = st["table"].long().gather(1, (begin // b).clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0]
    part, used = part[has], (begin % b)[has]
    _write(st["k"], st["ks"], k, page, slot, part, used, fmt, False)
    _write(st["v"], st["vs"], v, page, slot, part, used, fmt, True)
    if fmt == "e4m3":
        return _pool(st, q)
    _, page, slot = _places(st["start_all"], st["len"], st["rows_all"], b, st["table"])
    k, v = _gather_at(st, page, slot, torch.float32)
    return dict(q=q, k=k, v=v, ks=st["ks"], vs=st["vs"])


def _padded(codes, scales, table, fmt, order):
    """[S, H, keys, D] in fp32 of all pages of every sequence."""
    t = table.long()
    c = _as_numbers(codes[t], fmt) * scales[t][..., None, None]
    return c.permute(order).flatten(2, 3)


def _plain_attend(st):
    case = st["case"]
    fmt, h, grp, d = case["fmt"], case["heads"], case["group"], case["dim"]
    k = _padded(st["k"], st["ks"], st["table"], fmt, (0, 2, 1, 3, 4))
    v = _padded(st["v"], st["vs"], st["table"], fmt, (0, 2, 1, 4, 3))
    seqs, most, rows = case["seqs"], st["most"], st["rows"]
    n = (st["start"][1:] - st["start"][:-1]).long()
    i = torch.arange(most, device=k.device)
    at = (st["start"][:-1].long()[:, None] + i).clamp(max=rows - 1)
    q = st["q"].float()[at].view(seqs, most, h, grp, d).permute(0, 2, 3, 1, 4)
    t = torch.matmul(q.reshape(seqs, h, grp * most, d), k.transpose(2, 3).contiguous()) * st["scale"]
    if case["softcap"]:
        t = case["softcap"] * torch.tanh(t / case["softcap"])
    pos = (st["len"].long() - n)[:, None] + i
    j = torch.arange(k.shape[2], device=k.device)
    see = (j <= pos[..., None]) & (j < st["len"][:, None, None])
    if case["window"]:
        see &= j > pos[..., None] - case["window"]
    t = t.view(seqs, h, grp, most, -1).masked_fill_(~see[:, None, None], -math.inf)
    top = t.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (t - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, h, grp * most, -1), v).view(seqs, h, grp, most, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    real = i[None] < n[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, h * grp, d)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, most, h * grp)[real]
    return o.to(torch.bfloat16), lse.contiguous()


def run(state):
    if own:
        return _own_run(state)
    case, op = state["case"], state["case"]["op"]
    if op == "rope":
        return _rotate(state["x"], state["pos"], state["freq"], state["factor"],
                       case["interleaved"])
    if op == "append":
        return _plain_append(state)
    if op == "read":
        return _gather(state, torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    return _plain_attend(state)


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_rope(x, pos, freq, factor, interleaved):
    """Each pair as a complex number times factor * e^(i a)."""
    rot = 2 * freq.numel()
    angle = pos.double().outer(freq)
    turn = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    y = x.double().clone()
    one = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    two = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_code(x, fmt):
    """The nearest of all codes to each quotient; of two equally near ones the even one."""
    if fmt == "int8":
        low = x.floor()
        up = (x - low > 0.5) | ((x - low == 0.5) & (low % 2 != 0))
        return (low + up.double()).clamp(-127, 127)
    every = torch.arange(0, 127, device=x.device, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (every[1:] + every[:-1]) / 2
    a = x.abs()
    above = torch.searchsorted(mid, a, right=True)
    below = torch.searchsorted(mid, a, right=False)
    return torch.copysign(every[torch.where(above % 2 == 0, above, below)], x)


def _exact_append(st):
    case = st["case"]
    fmt, b, h = case["fmt"], case["block"], case["heads"]
    n, length = _lengths(case)
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    pool_k = st["k"].view(kind).float().double()
    pool_v = st["v"].view(kind).float().double().transpose(2, 3).contiguous()
    ks, vs = st["ks"].clone(), st["vs"].clone()
    at, q = 0, []
    for s in range(case["seqs"]):
        if not n[s]:
            continue
        rows = slice(at, at + n[s])
        at += n[s]
        pos = torch.arange(length[s] - n[s], length[s], device=DEV)
        k, v = st["new_k"][rows].double(), st["new_v"][rows].double()
        if case["rot"]:
            k = _exact_rope(k, pos, st["freq"], st["factor"], False)
        if st["q"] is not None:
            one = st["q"][rows].double()
            q.append(_exact_rope(one, pos, st["freq"], st["factor"], False) if case["rot"] else one)
        k, v = (t.float().to(torch.bfloat16).double() for t in (k, v))
        for first in range((length[s] - n[s]) // b * b, length[s], b):
            page = int(st["table"][s, first // b])
            lo = max(first, length[s] - n[s])
            hi = min(first + b, length[s])
            for pool, scales, x in ((pool_k, ks, k), (pool_v, vs, v)):
                x = x[lo - length[s] + n[s]:hi - length[s] + n[s]].transpose(0, 1)
                s_new = (x.abs().amax((1, 2)).float() / QMAX[fmt])
                s_new = s_new * (s_new >= MIN_SCALE)
                if lo > first:
                    s_old = scales[page]
                    s_new = torch.maximum(s_old, s_new)
                    e = pool[page, :, :lo - first]
                    pool[page, :, :lo - first] = torch.where(
                        (s_new > s_old)[:, None, None],
                        _exact_code(e * s_old.double()[:, None, None]
                                    / s_new.double().clamp(min=1e-300)[:, None, None], fmt), e)
                scales[page] = s_new
                pool[page, :, lo - first:hi - first] = _exact_code(
                    x / s_new.double()[:, None, None].masked_fill(s_new[:, None, None] == 0, math.inf), fmt)
    q = torch.cat(q) if st["q"] is not None else None
    if fmt == "e4m3":
        return dict(q=q, k=pool_k, v=pool_v.transpose(2, 3).contiguous(), ks=ks.double(), vs=vs.double())
    k, v = _exact_read(st, pool_k, pool_v, ks, vs, length, length)
    return dict(q=q, k=k, v=v, ks=ks.double(), vs=vs.double())


def _exact_read(st, pool_k, pool_v, ks, vs, n, length):
    """The last n tokens of each sequence; pools [pages, heads, block, dim] of numbers."""
    k, v, b = [], [], st["case"]["block"]
    for s, count in enumerate(n):
        if not count:
            continue
        pages = st["table"][s, :-(-length[s] // b)].long()
        for got, pool, scales in ((k, pool_k, ks), (v, pool_v, vs)):
            t = pool[pages] * scales[pages].double()[..., None, None]
            got.append(t.transpose(1, 2).flatten(0, 1)[length[s] - count:length[s]])
    return torch.cat(k), torch.cat(v)


def _exact_attend(st):
    case = st["case"]
    h, grp = case["heads"], case["group"]
    n, length = _lengths(case)
    kind = torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8
    out, lse, at = [], [], 0
    for s in range(case["seqs"]):
        if not n[s]:
            continue
        q = st["q"][at:at + n[s]].double()
        at += n[s]
        pages = st["table"][s, :-(-length[s] // case["block"])].long()
        p = (torch.arange(n[s], device=DEV) + length[s] - n[s])[:, None]
        j = torch.arange(length[s], device=DEV)[None]
        hidden = j > p
        if case["window"]:
            hidden = hidden | (j <= p - case["window"])
        o_s, l_s = [], []
        for head in range(h):
            k = st["k"][pages, head].view(kind).float().double() * st["ks"][pages, head].double()[:, None, None]
            v = st["v"][pages, head].view(kind).float().double() * st["vs"][pages, head].double()[:, None, None]
            k, v = k.flatten(0, 1)[:length[s]], v.transpose(1, 2).flatten(0, 1)[:length[s]]
            for g in range(grp):
                t = q[:, head * grp + g] @ k.T * st["scale"]
                if case["softcap"]:
                    t = torch.tanh(t / case["softcap"]) * case["softcap"]
                t = t.masked_fill(hidden, -math.inf)
                l_s.append(torch.logsumexp(t, 1))
                o_s.append(torch.exp(t - l_s[-1][:, None]) @ v)
        out.append(torch.stack(o_s, 1))
        lse.append(torch.stack(l_s, 1))
    return torch.cat(out), torch.cat(lse)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(st["x"], st["pos"], st["freq"], st["factor"], case["interleaved"])
    if op == "append":
        return _exact_append(st)
    if op == "read":
        kind = torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8
        k, v = (st[a].view(kind).float().double() for a in "kv")
        n, length = _lengths(case)
        return _exact_read(st, k, v.transpose(2, 3), st["ks"], st["vs"], n, length)
    return _exact_attend(st)
