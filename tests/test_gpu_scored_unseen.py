"""What no row sees may hold anything, wherever it lies: keys between the documents of a row, keys that the call's causal
rule hides from rows whose intervals reach them, keys that scattered intervals leave out; rows without keys.  And a NaN
in a key that some rows see stays in the forward with the blocks that see it."""
import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads
from oracle import scored as so
from tests.parity import to_np
from tests.test_gpu_scored import _i32, _slopes, _status_ok, _within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _documents(B, S, cu, prefix, causal=True, window=0):
    return so.row_bounds(B, S, S, causal, window, cu, prefix)


def _rows(B, Sq, f):
    lo, hi = np.zeros((B, Sq), np.int64), np.zeros((B, Sq), np.int64)
    for b in range(B):
        for i in range(Sq):
            lo[b, i], hi[b, i] = f(b, i)
    return lo, hi


def _scattered(B, Sq, Sk, seed):
    rng = np.random.RandomState(seed)
    lo = rng.randint(0, Sk // 6, (B, Sq)) * 6
    return lo, lo + rng.randint(0, 5, (B, Sq))  # never the last key of six


# name: (B, Sq, Sk, causal of the call, intervals)
MASKS = {
    # rows that see everything up to themselves, and padding behind them: the intervals reach into it
    "rule": lambda: (1, 300, 300, True, _rows(1, 300, lambda b, i: (0, 300) if i < 200 else (0, 0))),
    "rule_front": lambda: (2, 400, 400, True, _rows(2, 400, lambda b, i: (0, 400) if 130 < i < 140 + 150 * b else (0, 0))),
    # intervals that lie behind their rows' positions are empty under the rule
    "rule_ahead": lambda: (1, 390, 390, True, _rows(1, 390, lambda b, i: (i + 20, i + 60) if i % 3 else (i // 2, i - 5))),
    "between": lambda: (2, 420, 420, False, _documents(2, 420, [0, 100, 180, 300, 303, 420, 500, 560, 800, 840],
                                                       [0, -1, 20, -1, 0, -1, 0, -1, 5])),
    "between_both_ways": lambda: (1, 300, 300, False, _documents(1, 300, [0, 100, 120, 300], [0, -1, 0], causal=False)),
    "between_windows": lambda: (1, 700, 700, True, _documents(1, 700, [0, 90, 110, 400, 450, 700], [0, -1, 0, -1, 3], window=33)),
    "scattered": lambda: (2, 300, 300, False, _scattered(2, 300, 300, 1)),
    "scattered_rule": lambda: (1, 300, 420, True, _scattered(1, 300, 420, 2)),
    # a gap that only the two tiles of a pair together have, in both orders
    "pairs": lambda: (1, 512, 512, False, _rows(1, 512, lambda b, i: [(0, 100), (300, 400), (410, 500), (20, 99)][i // 128])),
    # the first tile's rows see everything, the next ones' only keys in front of their own: a gap under the rule alone
    "pairs_rule": lambda: (1, 512, 512, True, _rows(1, 512, lambda b, i: (0, 512) if i < 128 else
                                                   (140, 145) if i < 256 else (0, 0) if i < 400 else (300, 512))),
    "own": lambda: (1, 500, 500, True, _rows(1, 500, lambda b, i: (i // 100 * 100, i // 100 * 100 + 90)
                                            if i % 100 < 90 else (0, 0))),
    # few rows with long keys, many heads on few keys: split over the GPU
    "long": lambda: (1, 60, 3000, False, _rows(1, 60, lambda b, i: (700, 1900) if i % 2 else (2000, 2900))),
    "long_rule": lambda: (1, 200, 2600, True, _rows(1, 200, lambda b, i: (100, 2600) if i < 90 else (0, 0))),
}


def _visible(Sq, Sk, causal, lo, hi):
    h = np.minimum(hi, np.arange(Sq) + Sk - Sq + 1) if causal else hi
    j = np.arange(Sk)
    return h, (j >= lo[..., None]) & (j < h[..., None])


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (3.0, True)])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (3, 3, 128), (12, 1, 64)])
@pytest.mark.parametrize("name", MASKS)
def test_what_no_row_sees_may_hold_anything(name, Hq, Hkv, d, garbage, cap, bias):
    B, Sq, Sk, causal, (lo, hi) = MASKS[name]()
    h, seen = _visible(Sq, Sk, causal, lo, hi)
    keys, rows = torch.from_numpy(~seen.any(1)), torch.from_numpy(~seen.any(2))
    assert bool(keys.any())
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=61, with_dout=True)
    sl = _slopes(Hq, 0.3) if bias else None
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.09, lo, h, cap, None if sl is None else sl.double().numpy(),
                  to_np(t["dout"]), bounds=True)
    for n, dead in (("q", rows), ("dout", rows), ("k", keys), ("v", keys)):
        t[n].masked_fill_(dead[:, None, :, None], garbage)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    how = dict(softcap=cap, slopes=None if sl is None else sl.to(DEV),
               plan=fa.fa_mask_plan(_i32(lo.tolist()), _i32(hi.tolist()), Sk))
    o, lse = fa.fa_fwd_scored(q, k, v, causal, 0.09, **how)
    o[rows[:, None].expand(B, Hq, Sq).to(DEV)] = garbage  # nor is O read there
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, causal, 0.09, **how)
    torch.cuda.synchronize()
    _status_ok()
    live = (~rows)[:, None, :, None].expand(o.shape)
    _within(o[live.to(DEV)], r["o"][live.numpy()], r["tol_o"][live.numpy()], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    for n, x in zip(("dq", "dk", "dv"), g):
        _within(x, r[n], r["tol_" + n], n)
        dead = rows if n == "dq" else keys
        assert float(x.masked_select(dead[:, None, :, None].to(DEV)).abs().sum()) == 0.0


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (1, 1)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (3.0, True)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_nan_stays_with_the_blocks_that_see_its_key(where, cap, bias, Hq, Hkv):
    # rows 0..255 look past keys 50..99 on both sides; rows 256.. see them
    S, d = 512, 64
    lo, hi = _rows(1, S, lambda b, i: ((0, 50) if i % 2 else (100, 300)) if i < 256 else (40, 120))
    t = workloads.random_qkv(1, Hq, Hkv, S, S, d, seed=62)
    sl = _slopes(Hq) if bias else None
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.1, lo, hi, cap, None if sl is None else sl.double().numpy(),
                  bounds=True)
    t[where][:, :, 70] = float("nan")
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=cap, slopes=None if sl is None else sl.to(DEV),
                              plan=fa.fa_mask_plan(_i32(lo.tolist()), _i32(hi.tolist()), S))
    torch.cuda.synchronize()
    _status_ok()
    assert bool(o[:, :, 256:].isnan().all())
    near = slice(0, 256)
    _within(o[:, :, near], r["o"][:, :, near], r["tol_o"][:, :, near], "O")
    _within(lse[:, :, near], r["lse"][:, :, near], r["tol_lse"][:, :, near], "LSE")
