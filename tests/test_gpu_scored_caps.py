"""Capped scores over the whole range of caps, forward, backward and decode, whole and masked tiles: the oracle's bounds
do not grow with the cap (a score is off by what its own size allows, or by 2^-22 of 256)."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads
from oracle import scored as so
from tests.parity import to_np
from tests.test_gpu_scored import _i32, _run, _slopes, _status_ok, _within

pytestmark = pytest.mark.gpu
DEV = "cuda"

CAPS = [100.0, 256.0, 300.0, 1.0e3, 1.0e4, 1.0e5, 2.0 ** 18, 2.0 ** 20]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", CAPS)
def test_large_caps(cap, bias, d):
    sl = _slopes(4) if bias else None
    # rows 256 to 299 see whole tiles, all others a masked one as well
    _run(1, 4, 2, 300, 300, d, True, cap, sl, planned=False, seed=51)
    _run(2, 4, 2, 300, 300, d, True, cap, sl, 150, [0, 70, 300, 430, 600], [0, 130, -1, 40], seed=52)


@pytest.mark.parametrize("cap", [300.0, 1.0e3])
@pytest.mark.parametrize("planned", [False, True])
def test_scores_of_every_size_beside_each_other(cap, planned):
    # rows whose scores reach past a large cap lie in one warp with rows of ordinary ones
    B, Hq, Hkv, S, d = 1, 2, 1, 300, 64
    t = workloads.random_qkv(B, Hq, Hkv, S, S, d, seed=53, with_dout=True)
    t["q"][:, :, ::7] *= 1.5 * cap
    t["q"][:, :, 3::14] *= 0.3 * cap
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    lo, hi = so.row_bounds(B, S, S, True)
    plan = fa.fa_mask_plan(*fa.fa_row_bounds(B, S, S, True), S) if planned else None
    how = dict(softcap=cap, plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, not planned, 0.125, **how)
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, not planned, 0.125, **how)
    torch.cuda.synchronize()
    _status_ok()
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.125, lo, hi, cap, None, to_np(t["dout"]), bounds=True)
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    for n, x in zip(("dq", "dk", "dv"), g):
        _within(x, r[n], r["tol_" + n], n)


@pytest.mark.parametrize("cap,scale,mult", [(50.0, 2.0 ** -14, 2048.0), (2.0 ** 20, 2.0 ** -14, 2048.0), (2.0 ** 20, 0.0, 1.0),
                                            (1.0, 2.0 ** -70, 1.0), (2.0 ** 20, 200.0, 2.0 ** -11)])
def test_scales_far_from_one(cap, scale, mult):
    _run(1, 2, 1, 200, 200, 64, True, cap, None, planned=False, scale=scale, mult=mult, seed=54)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("cap", CAPS)
def test_decode_under_large_caps(cap, Hq, Hkv, d):
    lens, room = [700, 1, 333], 700
    t = workloads.random_qkv(3, Hq, Hkv, 1, room, d, seed=55)
    t["q"][1:] *= 8
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_decode_scored(t["q"].to(DEV), t["k"].to(DEV), t["v"].to(DEV), _i32(lens), scale, softcap=cap)
    torch.cuda.synchronize()
    _status_ok()
    for b, n in enumerate(lens):
        r = so.attend(to_np(t["q"][b:b + 1]), to_np(t["k"][b:b + 1, :, :n]), to_np(t["v"][b:b + 1, :, :n]), scale,
                      np.array([[0]]), np.array([[n]]), cap, bounds=True)
        # the decode keeps weights in two terms: nothing of the oracle's 2^-8 for them, only O's own rounding
        tol = 2.0 ** -8 * np.abs(r["o"]) + (r["tol_lse"][..., None] * 4 + 2.0 ** -14) * np.abs(to_np(t["v"][b, :, :n])).max()
        _within(o[b:b + 1], r["o"], tol, f"O {b}")
        _within(lse[b:b + 1, :, None], r["lse"], r["tol_lse"], f"LSE {b}")
