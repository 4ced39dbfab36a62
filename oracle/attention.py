"""Float64 oracle of the rotary positions, the 8-bit key/value cache and the
attention over it, one token and one head at a time, from the definitions:

  rope    (x1, x2) -> factor (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
          a = position * freq[pair]; rounded to fp32, then to bf16
  cache   per page and head: scale = amax * fl32(1/Q) (Q = 127 or 448), never
          smaller while the page holds earlier tokens; codes = round(x / scale),
          nearest, ties to even
  attend  softmax over the keys a query sees, in the order of the definition
"""

from __future__ import annotations

import numpy as np

from .matquant import bf16_round

MIN_SCALE = 2.0 ** -100
QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3_values() -> np.ndarray:
    """The 127 non-negative numbers of the format (sign, 4 exponent bits of
    bias 7, 3 mantissa bits; no infinity, the pattern 0x7f is NaN)."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = e4m3_values()


def numbers(codes: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 codes -> the numbers they stand for, in float64."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    return table[codes]


def round_codes(x: np.ndarray, fmt: str) -> np.ndarray:
    """Quotients to uint8 codes: nearest, ties to even, saturating, NaN to 0."""
    x = np.where(np.isnan(x), 0.0, np.asarray(x, dtype=np.float64))
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    i = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 125)  # E4M3[i] <= a
    lo, hi = a - E4M3[i], E4M3[i + 1] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 1))
    code = (i + up).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def rope_turn(x, pos, freq, factor=1.0, interleaved=False) -> np.ndarray:
    """x [T, H, D], pos [T] -> float64 [T, H, D], not rounded."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = len(freq)
    for i in range(half):
        a = np.asarray(pos, dtype=np.float64) * freq[i]
        c, s = (np.cos(a) * factor)[:, None], (np.sin(a) * factor)[:, None]
        i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[:, :, i1] = x[:, :, i1] * c - x[:, :, i2] * s
        out[:, :, i2] = x[:, :, i2] * c + x[:, :, i1] * s
    return out


def to_bf16(x) -> np.ndarray:
    """float64 -> fp32 -> bf16 values (as float64); NaN and infinities kept."""
    with np.errstate(over="ignore", invalid="ignore"):
        f = np.asarray(x).astype(np.float32)
        fin = np.isfinite(f)
        r = bf16_round(np.where(fin, f, 0.0).astype(np.float32)).astype(np.float64)
    return np.where(fin, r, f.astype(np.float64))


class Cache:
    """k codes [P, H, B, D], v codes [P, H, D, B], scales fp32 [P, H]."""

    def __init__(self, k, v, ks, vs, fmt):
        self.k, self.v, self.ks, self.vs, self.fmt = k.copy(), v.copy(), ks.copy(), vs.copy(), fmt
        self.pages, self.heads, self.block, self.dim = k.shape

    def _page(self, table, s, pos):
        pi = pos // self.block
        if pos < 0 or pi >= table.shape[1]:
            return -1
        p = int(table[s, pi])
        return p if 0 <= p < self.pages else -1

    def _put(self, codes, scales, page, head, used, x):
        """New values x [n, D] at places used .. of a page's codes [B, D]."""
        fin = np.abs(x[np.isfinite(x)])
        amax = np.float32(fin.max()) if fin.size else np.float32(0)
        fresh = np.float32(amax * np.float32(np.float32(1) / np.float32(QMAX[self.fmt])))
        if fresh < MIN_SCALE:
            fresh = np.float32(0)
        now = fresh
        if used:
            was = scales[page, head]
            now = max(was, fresh)
            if now > was:
                old = numbers(codes[:used], self.fmt)
                codes[:used] = round_codes(old * float(was) / float(now), self.fmt)
        scales[page, head] = now
        if now > 0:
            with np.errstate(invalid="ignore"):
                codes[used:used + len(x)] = round_codes(x / float(now), self.fmt)
        else:
            codes[used:used + len(x)] = 0

    def append(self, q_start, kv_len, table, k, v):
        """k, v: the bf16 values [rows, H, D] as float64."""
        for s in range(len(kv_len)):
            r0, n = int(q_start[s]), int(q_start[s + 1] - q_start[s])
            start = int(kv_len[s]) - n
            i = 0
            while i < n:
                pos = start + i
                m = min(n - i, self.block - pos % self.block)
                page = self._page(table, s, pos)
                if page >= 0:
                    used = pos % self.block
                    for h in range(self.heads):
                        self._put(self.k[page, h], self.ks, page, h, used, k[r0 + i:r0 + i + m, h])
                        vt = np.ascontiguousarray(self.v[page, h].T)
                        self._put(vt, self.vs, page, h, used, v[r0 + i:r0 + i + m, h])
                        self.v[page, h] = vt.T
                i += m

    def token(self, table, s, pos):
        """(k, v) float64 [H, D] of a position, or None where none is held."""
        page = self._page(table, s, pos)
        if page < 0:
            return None
        t = pos % self.block
        k = numbers(self.k[page, :, t], self.fmt) * self.ks[page].astype(np.float64)[:, None]
        v = numbers(np.ascontiguousarray(self.v[page, :, :, t]), self.fmt) * \
            self.vs[page].astype(np.float64)[:, None]
        return k, v

    def read(self, q_start, kv_len, table, rows):
        """k, v [rows, H, D]; rows beyond the last sequence are NaN."""
        k = np.full((rows, self.heads, self.dim), np.nan)
        v = k.copy()
        for s in range(len(kv_len)):
            for r in range(int(q_start[s]), int(q_start[s + 1])):
                got = self.token(table, s, int(kv_len[s]) - int(q_start[s + 1]) + r)
                k[r], v[r] = got if got is not None else (0.0, 0.0)
        return k, v

    def attend(self, q_start, kv_len, table, q, scale, softcap=0.0, window=0, causal=True):
        """out [rows, Hq, D], lse [rows, Hq] and, for error bounds, per output
        entry sum_j p_j |v_j|, per row the largest sum_d |scale q_d k_jd|, the
        number of keys seen and the largest |v|."""
        rows, hq, d = q.shape
        grp = hq // self.heads
        out, lse = np.full((rows, hq, d), np.nan), np.full((rows, hq), np.nan)
        mass, size = np.zeros((rows, hq, d)), np.zeros((rows, hq))
        seen, vmax = np.zeros((rows, hq)), np.zeros((rows, hq))
        for s in range(len(kv_len)):
            held = {}
            for j in range(max(0, int(kv_len[s]))):
                t = self.token(table, s, j)
                if t is not None:
                    held[j] = t
            js = np.array(sorted(held), dtype=np.int64)
            for r in range(int(q_start[s]), int(q_start[s + 1])):
                pos = int(kv_len[s]) - int(q_start[s + 1]) + r
                see = js[js <= pos] if causal else (js if pos >= 0 else js[:0])
                if window:
                    see = see[see > pos - window]
                if not len(see):
                    out[r], lse[r] = 0.0, -np.inf
                    continue
                k = np.stack([held[j][0] for j in see], 1)  # [H, n, D]
                v = np.stack([held[j][1] for j in see], 1)
                for h in range(hq):
                    kk, vv = k[h // grp], v[h // grp]
                    t = kk @ q[r, h] * scale
                    size[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max() * abs(scale)
                    if softcap:
                        t = softcap * np.tanh(t / softcap)
                    m = t.max()
                    p = np.exp(t - m)
                    lse[r, h] = m + np.log(p.sum())
                    out[r, h] = p @ vv / p.sum()
                    mass[r, h] = p @ np.abs(vv) / p.sum()
                    seen[r, h], vmax[r, h] = len(see), np.abs(vv).max()
        return out, lse, dict(mass=mass, size=size, seen=seen, vmax=vmax)
