"""Plain 64-bit definitions of the paged 8-bit KV cache operators (NumPy): block
tables and slot maps, the quantising write, the dequantising read, block
selection, and attention over the cache.  Loops over requests, runs and heads;
no code is shared with the GPU path."""
from __future__ import annotations

import math

import numpy as np


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = -v if c & 128 else v
    return t


E4M3 = _e4m3_table()


def decode_codes(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (ties to the even code), magnitudes above 448 and
    infinities to 448, NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=448.0), 448.0)
    pos = E4M3[:127]
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = pos[hi] - a, a - pos[lo]
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def power_of_two_scale(amax: float, top: float, lowest=-100, highest=119) -> float:
    """The smallest 2^e with amax <= top * 2^e, e in [lowest, highest]."""
    if not amax > 0:
        return 2.0 ** lowest
    m, e = math.frexp(amax / top)
    return 2.0 ** min(max(e - (m == 0.5), lowest), highest)


def pages_of(n: int, ps: int) -> int:
    return -(-n // ps)


def assign(seqlens, newlens, ps, table, free, total_new):
    """(table, slots, cu_new, seqlens_out, cu_k, n_used)."""
    table = np.array(table, np.int64)
    slots = np.full(total_new, -1, np.int64)
    asked = used = at = 0
    out, cu = [], [0]
    for b, (n, m) in enumerate(zip(seqlens, newlens)):
        n, m = max(int(n), 0), max(int(m), 0)
        have, full = pages_of(n, ps), pages_of(n + m, ps)
        ok = full <= table.shape[1] and at + m <= total_new
        if ok:
            asked += full - have
            if full > have and asked > len(free):
                ok = False
        if ok:
            for j in range(have, full):
                table[b, j] = free[asked - full + j]
                used = asked
            for i in range(m):
                page = table[b, (n + i) // ps]
                slots[at + i] = page * ps + (n + i) % ps if page >= 0 else -1
        out.append(n + m if ok else n)
        at += m
        cu.append(at)
    return table, slots, np.array(cu), np.array(out), np.array([0] + list(np.cumsum(out))), used


class Cache:
    """codes uint8 [2][pages,Hkv,ps,d] (K, V), scales [2][pages,Hkv], bounds [pages,Hkv,2,d]."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, bounds=None):
        self.codes = [np.array(k_codes), np.array(v_codes)]
        self.scale = [np.array(k_scale, np.float64), np.array(v_scale, np.float64)]
        self.bounds = None if bounds is None else np.array(bounds, np.int64)

    def write(self, k, v, slots):
        """k, v [Hkv, n, d] float64."""
        pages, heads, ps, _ = self.codes[0].shape
        t = 0
        while t < len(slots):
            s = int(slots[t])
            if not 0 <= s < pages * ps:
                t += 1
                continue
            end = t + 1
            while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % ps:
                end += 1
            for which, x in enumerate((k, v)):
                for h in range(heads):
                    self._run(which, h, s // ps, s % ps, x[h, t:end])
            t = end

    def _run(self, which, h, page, off, x):
        codes, scale = self.codes[which], self.scale[which]
        a = np.abs(x)
        tok = power_of_two_scale(float(a[np.isfinite(a)].max(initial=0.0)), 448.0)
        was = float(scale[page, h]) if off else 0.0
        now = max(was, tok)
        r = was / now
        if off and now > was:
            codes[page, h, :off] = encode(E4M3[codes[page, h, :off]] * r)
        new = encode(x / now)
        codes[page, h, off:off + len(x)] = new
        scale[page, h] = now
        if which == 0 and self.bounds is not None:
            y = np.nan_to_num(E4M3[new], nan=0.0) / 4
            hi, lo = np.ceil(y.max(axis=0)), np.floor(y.min(axis=0))
            if off:
                top, low = self.bounds[page, h, 0] * r, self.bounds[page, h, 1] * r
                hi, lo = np.maximum(hi, np.ceil(top)), np.minimum(lo, np.floor(low))
                if math.frexp(r)[0] != 0.5:  # held codes are rounded too
                    hi = np.maximum(hi, np.ceil(E4M3[encode(4 * top)] / 4))
                    lo = np.minimum(lo, np.floor(E4M3[encode(4 * low)] / 4))
            self.bounds[page, h] = np.stack([hi, lo])

    def values(self, which, page, h):
        return E4M3[self.codes[which][page, h]] * self.scale[which][page, h]

    def gather(self, which, table_row, h, positions):
        """Values [n, d] at the positions; absent[n] where the block has no page."""
        pages, _, ps, d = self.codes[0].shape
        out, absent = np.zeros((len(positions), d)), np.zeros(len(positions), bool)
        for i, j in enumerate(positions):
            blk = j // ps
            page = int(table_row[blk]) if blk < len(table_row) else -1
            if 0 <= page < pages:
                out[i] = E4M3[self.codes[which][page, h, j % ps]] * self.scale[which][page, h]
            else:
                absent[i] = True
        return out, absent


def bounds_of_codes(codes: np.ndarray) -> np.ndarray:
    """int bounds [pages,Hkv,2,d] of whole pages of codes."""
    y = np.nan_to_num(E4M3[codes], nan=0.0) / 4
    return np.stack([np.ceil(y.max(axis=2)), np.floor(y.min(axis=2))], axis=2).astype(np.int64)


def select(q, bounds, k_scale, table, seqlens, ps, k_blocks, n_first, n_last):
    """q [B,Hq,Sq,d] float64.  Returns (sel, n_sel)."""
    B, Hq, Sq, d = q.shape
    pages, heads = k_scale.shape
    room = table.shape[1]
    sel = np.full((B, heads, k_blocks), -1, np.int64)
    n_sel = np.zeros((B, heads), np.int64)
    for b in range(B):
        n = pages_of(min(max(int(seqlens[b]), 0), room * ps), ps)
        for h in range(heads):
            rows = q[b, h * (Hq // heads):(h + 1) * (Hq // heads)].reshape(-1, d)
            score = np.full(n, -np.inf)
            for row in rows:
                s = power_of_two_scale(float(np.abs(row).max()), 127.0)
                w = np.clip(np.rint(row / s), -127, 127)
                for i in range(n):
                    page = int(table[b, i])
                    if 0 <= page < pages:
                        u = np.maximum(w * bounds[page, h, 0], w * bounds[page, h, 1]).sum()
                        score[i] = max(score[i], u * float(k_scale[page, h]) * s * 4)
            score[:n_first] = np.inf
            score[max(n - n_last, 0):] = np.inf
            got = np.sort(np.argsort(-score, kind="stable")[:k_blocks])
            sel[b, h, :len(got)] = got
            n_sel[b, h] = len(got)
    return sel, n_sel


def attend(q, cache: Cache, table, seqlens, scale, sel=None, n_sel=None):
    """q [B,Hq,Sq,d] float64.  Returns (o, lse, spread, score_size, v_top): spread is
    sum_j w_j |v_j| per output, score_size the largest scale * sum_i |q_i k_i| of a
    row's visible keys, v_top the largest magnitude that the V scales of the row's
    keys allow (they enter the rounding bounds of a test)."""
    B, Hq, Sq, d = q.shape
    heads, ps = cache.codes[0].shape[1:3]
    room = table.shape[1] * ps
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    v_top = np.zeros(q.shape[:3])
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), room)
        for h in range(heads):
            if sel is None:
                pos = np.arange(n)
            else:
                blocks = [int(i) for i in sel[b, h, :max(int(n_sel[b, h]), 0)]]
                pos = np.array([i * ps + j for i in blocks if 0 <= i < pages_of(n, ps)
                                for j in range(ps) if i * ps + j < n], np.int64)
            k, absent = cache.gather(0, table[b], h, pos)
            v, _ = cache.gather(1, table[b], h, pos)
            used = {int(table[b, j // ps]) for j, a in zip(pos, absent) if not a}
            top = 448.0 * max((float(cache.scale[1][page, h]) for page in used), default=0.0)
            v_top[b, h * (Hq // heads):(h + 1) * (Hq // heads)] = top
            for g in range(h * (Hq // heads), (h + 1) * (Hq // heads)):
                for i in range(Sq):
                    see = ~absent & (pos <= i + n - Sq)
                    if not see.any():
                        continue
                    x = k[see] @ q[b, g, i] * scale
                    m = x.max()
                    w = np.exp(x - m)
                    lse[b, g, i] = m + math.log(w.sum()) if not math.isnan(m) else math.nan
                    w /= w.sum()
                    o[b, g, i] = w @ v[see]
                    spread[b, g, i] = w @ np.abs(v[see])
                    size[b, g, i] = (np.abs(k[see]) @ np.abs(q[b, g, i])).max() * scale
    return o, lse, spread, size, v_top
