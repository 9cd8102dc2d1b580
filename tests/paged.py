"""Shared helpers of the paged-cache tests: seeded caches and requests, and the
rounding bounds of an attention output."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as po

DEV = "cuda"


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn_bf16(gen, *shape, mult=1.0):
    return (torch.randn(*shape, generator=gen) * mult).to(torch.bfloat16)


def make_cache(seed, pages, heads, ps, d, spread=0.3):
    """A filled cache (CPU tensors) and its oracle."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn(pages, heads, ps, d, generator=gen) * torch.exp(
            spread * torch.randn(pages, heads, 1, d, generator=gen))
        x = x.double().numpy()
        scale = np.array([[po.power_of_two_scale(np.abs(x[p, h]).max(), 448.0)
                           for h in range(heads)] for p in range(pages)])
        out.append((po.encode(x / scale[:, :, None, None]), scale))
    (kc, ks), (vc, vs) = out
    return po.Cache(kc, vc, ks, vs, po.bounds_of_codes(kc))


def on_gpu(cache):
    """k_cache, v_cache, k_scale, v_scale, k_bounds as CUDA tensors."""
    t = [torch.from_numpy(np.array(c)).to(DEV) for c in cache.codes]
    t += [torch.from_numpy(s.astype(np.float32)).to(DEV) for s in cache.scale]
    t.append(torch.from_numpy(cache.bounds.astype(np.int8)).to(DEV))
    return t


def make_table(seed, lens, ps, pages, room=None):
    """Block tables [B, room] over distinct shuffled pages, -1 behind the last block."""
    order = np.random.RandomState(seed).permutation(pages)
    room = room or max(1, max(po.pages_of(max(n, 0), ps) for n in lens))
    table, at = np.full((len(lens), room), -1, np.int32), 0
    for b, n in enumerate(lens):
        m = min(po.pages_of(max(n, 0), ps), room)
        table[b, :m] = order[at:at + m]
        at += m
    assert at <= pages
    return table


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def attention_bounds(ref_o, ref_lse, spread, size, v_top, n_keys, d):
    """Element-wise bounds of O and LSE against the 64-bit values.

    A score is a sum of d products in fp32 (each term off by at most (d + 4) *
    2^-24 of sum |q k|, scaling included): a weight is off by twice that,
    relatively.  A weight is rounded to f16 (half a step: 2^-11) and its exponential
    is off by 2^-21.  Sums over the keys run in fp32: n * 2^-24.  O is rounded to bf16
    (half a step: 2^-8).  The LSE sees the score's error, the sum's and its own
    rounding to fp32.

    A weight is stored in f16 as w * 2^9 * (its page's V scale / the largest one): below
    f16's normal range its rounding is at most 2^-25 there, 2^-34 of the largest
    weight and V scale, so each key adds at most 2^-34 * v_top (the normaliser is at
    least 1: the key that set the running maximum counts 1)."""
    eps = 2.0 ** -24
    score = (d + 4) * eps * size
    rel = 2 * score + 2.0 ** -11 + 2.0 ** -21 + n_keys * eps
    tol_o = 2.0 ** -8 * np.abs(ref_o) + rel[..., None] * spread * (1 + 2.0 ** -8) + (
        n_keys * 2.0 ** -34 * v_top[..., None])
    tol_lse = score + (n_keys + 8) * eps + 2.0 ** -21 + 4 * eps * np.abs(
        np.where(np.isfinite(ref_lse), ref_lse, 0.0))
    return tol_o, tol_lse


def check_attention(o, lse, ref, n_keys, d):
    ref_o, ref_lse, spread, size, v_top = ref
    got_o, got_l = f64(o), f64(lse)
    assert np.array_equal(np.isnan(got_o), np.isnan(ref_o)), "NaN pattern of O"
    assert np.array_equal(np.isnan(got_l), np.isnan(ref_lse)), "NaN pattern of LSE"
    dead = ref_lse == -np.inf
    assert np.array_equal(got_l == -np.inf, dead), "-inf pattern of LSE"
    assert np.all(got_o[dead] == 0.0)
    live = ~dead & ~np.isnan(ref_lse)
    tol_o, tol_l = attention_bounds(ref_o, ref_lse, spread, size, v_top, n_keys, d)
    fine = live[..., None] & ~np.isnan(ref_o)
    if fine.any():
        worst = (np.abs(got_o[fine] - ref_o[fine]) / tol_o[fine]).max()
        assert worst <= 1.0, f"O is off by {worst:.2f} of its bound"
    if live.any():
        worst = (np.abs(got_l[live] - ref_lse[live]) / tol_l[live]).max()
        assert worst <= 1.0, f"LSE is off by {worst:.2f} of its bound"
