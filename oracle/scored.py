"""Attention with capped and biased scores under row intervals, head norms with rotation, and the intervals
themselves, in plain numpy FP64: full score matrices, no tiling, and no code shared with the GPU path.

With ``bounds=True`` the attention also gives, element by element, how far a computation may be off that rounds
where the library documents it does: weights and score gradients to bf16 for their products (half a step is 2^-8
of the value), O and the gradients to bf16 at the end, everything else in fp32."""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8  # half a step of bf16, relative to the value
F32 = 2.0 ** -24


def row_bounds(B, Sq, Sk, causal, window=0, cu=None, prefix=None):
    """lo, hi [B, Sq], by the definition, one row at a time."""
    lo, hi = np.zeros((B, Sq), np.int64), np.zeros((B, Sq), np.int64)
    for b in range(B):
        for i in range(Sq):
            p = i + Sk - Sq
            start, end, pre = 0, Sk, 0
            if cu is not None:
                at = [d for d in range(len(cu) - 1) if cu[d] <= b * Sk + p < cu[d + 1]]
                if p < 0 or not at:
                    continue
                start, end = max(0, cu[at[0]] - b * Sk), min(Sk, cu[at[0] + 1] - b * Sk)
                pre = prefix[at[0]] if prefix is not None else 0
            elif prefix is not None:
                pre = prefix[b]
            if pre < 0:
                continue
            l, h = start, end
            if causal:
                h = min(h, max(p + 1, start + pre))
            if window:
                l = max(l, p - window + 1)
                if not causal:
                    h = min(h, p + window)
            if h > l:
                lo[b, i], hi[b, i] = l, h
    return lo, hi


def attend(q, k, v, scale, lo, hi, cap=0.0, slopes=None, dout=None, bounds=False):
    """o, lse (and dq, dk, dv with dout) of q [B,Hq,Sq,d], k, v [B,Hkv,Sk,d]; bounds adds tol_<name>."""
    B, Hq, Sq, d = q.shape
    Hkv, Sk = k.shape[1:3]
    group = Hq // Hkv
    p = np.arange(Sq) + Sk - Sq
    j = np.arange(Sk)
    r = dict(o=np.zeros_like(q), lse=np.full((B, Hq, Sq), -np.inf))
    if dout is not None:
        r.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    if bounds:
        r.update({"tol_" + n: np.zeros_like(x) for n, x in list(r.items())})
        r["tol_lse"][:] = 0.0
    for b in range(B):
        seen = (j[None] >= lo[b][:, None]) & (j[None] < hi[b][:, None])
        live = seen.any(1)
        if not live.any():
            continue
        for h in range(Hq):
            kk, vv, qq = k[b, h // group], v[b, h // group], q[b, h]
            s = np.where(seen, qq @ np.where(seen.any(0)[:, None], kk, 0).T * scale, 0.0)
            t = cap * np.tanh(s / cap) if cap else s
            slope = 0.0 if slopes is None else float(slopes[h])
            z = np.where(seen, t - slope * np.abs(p[:, None] - j[None]), -np.inf)
            m = np.where(live, z.max(1, initial=-np.inf), 0.0)
            e = np.exp(z - m[:, None])
            total = np.where(live, e.sum(1), 1.0)
            P = e / total[:, None]
            vv0 = np.where(seen.any(0)[:, None], vv, 0)
            kk0 = np.where(seen.any(0)[:, None], kk, 0)
            qq0 = np.where(live[:, None], qq, 0)
            r["o"][b, h] = P @ vv0
            r["lse"][b, h] = np.where(live, m + np.log(total), -np.inf)
            if bounds:
                # exponents: d products of a score added in fp32 in any order, the cap, the bias, the sum
                absS = np.where(seen, np.abs(qq0) @ np.abs(kk0).T * scale, 0.0)
                far = np.abs(p[:, None] - j[None]) * abs(slope)
                ez = (d + 8) * F32 * absS + 2.0 ** -20 * (np.abs(t) + far) + 2.0 ** -21 * min(cap, 256.0) + 2.0 ** -21
                ez = np.where(seen, ez, 0.0)
                el = (P * ez).sum(1) + Sk * F32 + 2.0 ** -20 * (1 + np.abs(np.where(live, r["lse"][b, h], 0)))
                r["tol_lse"][b, h] = el
                ew = 2 * (ez + el[:, None])  # relative error of a weight before rounding
                spread = (P * (BF16 * 2 + ew)) @ np.abs(vv0)  # the weights' and their sum's rounding
                tol_o = spread * (1 + BF16) + BF16 * np.abs(r["o"][b, h]) + 2.0 ** -100
                r["tol_o"][b, h] = tol_o
            if dout is None:
                continue
            do = np.where(live[:, None], dout[b, h], 0)
            dP = do @ vv0.T
            D = (do * r["o"][b, h]).sum(1)
            dz = P * (dP - D[:, None])
            g = 1 - np.tanh(s / cap) ** 2 if cap else 1.0
            ds = np.where(seen, dz * g, 0.0)
            r["dv"][b, h // group] += P.T @ do
            r["dq"][b, h] = ds @ kk0 * scale
            r["dk"][b, h // group] += ds.T @ qq0 * scale
            if bounds:
                eD = (np.abs(do) * tol_o).sum(1) + d * F32 * (np.abs(do) * np.abs(r["o"][b, h])).sum(1)
                edP = (d + 2) * F32 * (np.abs(do) @ np.abs(vv0).T)
                rel = ew + 2.0 ** -10 + (2.0 ** -20 if cap else 0)  # weight, f16 and the derivative
                eds = np.abs(ds) * (BF16 + rel) + P * (edP + eD[:, None]) * (1 + BF16 + rel)
                eds += 2.0 ** -39 * np.abs(dP - D[:, None]) * seen  # weights below 2^-29 lose bits in f16
                if cap:  # 1 - tanh^2 off by 2^-20 of 1
                    eds += np.abs(dz) * 2.0 ** -20
                n = Sq + Sk
                r["tol_dq"][b, h] = (eds + n * F32 * np.abs(ds)) @ np.abs(kk0) * scale
                r["tol_dk"][b, h // group] += (eds + n * F32 * np.abs(ds)).T @ np.abs(qq0) * scale
                r["tol_dv"][b, h // group] += (P * (BF16 + ew + n * F32)).T @ np.abs(do)
    if bounds and dout is not None:
        for n in ("dq", "dk", "dv"):
            r["tol_" + n] = r["tol_" + n] * (1 + BF16) + BF16 * np.abs(r[n]) + 2.0 ** -100
    return r


def _turn(x, angles, rot, interleaved, back=False):
    """x [..., d] with its first `rot` channels turned by angles [..., rot / 2]."""
    y = x.copy()
    c, s = np.cos(angles), np.sin(angles)
    if back:
        s = -s
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def angles(positions, inv_freq, freq_axis):
    """[B, S, 1, rot / 2] from positions [n_axes, B, S]; frequencies of axes that are not there do not turn."""
    n_axes, B, S = positions.shape
    out = np.zeros((B, S, 1, len(inv_freq)))
    for i, f in enumerate(inv_freq):
        ax = 0 if freq_axis is None else int(freq_axis[i])
        if ax < n_axes:
            # whole turns fall off in exact arithmetic: positions are whole numbers, f a float
            out[:, :, 0, i] = np.array([[float((int(n) * _turns(float(f))) % (1 << 200)) / (1 << 200) for n in row]
                                        for row in positions[ax]]) * 2 * np.pi
    return out


_PI_DIGITS = "3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982148"


def _turns(f):
    """f / (2 pi) in units of 2^-200, a whole number."""
    from fractions import Fraction
    pi = Fraction(int(_PI_DIGITS), 10 ** (len(_PI_DIGITS) - 1))
    return int(Fraction(f) / (2 * pi) * (1 << 200))


def norm_rope(x, w, w_off, eps, ang, rot, interleaved):
    """y [B, H, S, d] of x [B, S, H, d] (w None: no norm)."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + w_off)
    if rot:
        x = _turn(x, ang, rot, interleaved)
    return x.transpose(0, 2, 1, 3)


def norm_rope_bwd(x, w, w_off, eps, ang, rot, interleaved, dy):
    """dx [B, S, H, d], dw [d] (None without w) and, for tolerances, the size of what dx and dw are summed of."""
    g = dy.transpose(0, 2, 1, 3)
    if rot:
        g = _turn(g, ang, rot, interleaved, back=True)
    if w is None:
        return g, None, np.abs(g), None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    a = g * (w + w_off)
    dx = r * (a - n * (a * n).mean(-1, keepdims=True))
    size = r * (np.abs(a) + np.abs(n) * np.abs(a * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1, 2)), size, np.abs(g * n).sum((0, 1, 2))
