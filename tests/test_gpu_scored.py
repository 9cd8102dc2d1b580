"""GPU parity of attention on capped and biased scores under row intervals (fa_row_bounds, fa_mask_plan,
fa_fwd_scored, fa_bwd_scored, fa_decode_scored) against the FP64 oracle.  Tolerances are the oracle's own, element by
element: what rounding weights and score gradients to bf16 and everything else to fp32 may do to each output."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads
from oracle import scored as so
from tests.parity import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _status_ok():
    st, word = fa.fa_device_status()
    assert st == 0, hex(word)


def _within(got, ref, tol, what):
    got = to_np(got) if isinstance(got, torch.Tensor) else got
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(got)), f"{what}: finite where the reference is not, or the other way"
    assert np.array_equal(got[~fin], ref[~fin]), f"{what}: infinities differ"
    over = np.abs(got[fin] - ref[fin]) - tol[fin]
    assert not over.size or over.max() <= 0, (
        f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, worst by {over.max():.3e}")


def _slopes(H, steep=1.0):
    return torch.tensor([steep * 2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32)


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def _run(B, Hq, Hkv, Sq, Sk, d, causal, cap=0.0, slopes=None, window=0, cu=None, prefix=None, mult=1.0, seed=1,
         planned=True, back=True, scale=None):
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=seed, q_mult=mult, with_dout=True)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    lo, hi = so.row_bounds(B, Sq, Sk, causal, window, cu, prefix)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    sl = None if slopes is None else slopes.to(DEV)
    plan, ca = None, causal
    if planned:
        gl, gh = fa.fa_row_bounds(B, Sq, Sk, causal, window=window, cu_docs=_i32(cu), prefix=_i32(prefix))
        assert np.array_equal(gl.cpu().numpy(), lo) and np.array_equal(gh.cpu().numpy(), hi)
        plan, ca = fa.fa_mask_plan(gl, gh, Sk), False
    o, lse = fa.fa_fwd_scored(q, k, v, ca, scale, softcap=cap, slopes=sl, plan=plan)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), scale, lo, hi, float(np.float32(cap)),
                  None if slopes is None else slopes.double().numpy(), to_np(t["dout"]), bounds=True)
    torch.cuda.synchronize()
    _status_ok()
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    if back:
        g = fa.fa_bwd_scored(q, k, v, o, do, lse, ca, scale, softcap=cap, slopes=sl, plan=plan)
        torch.cuda.synchronize()
        _status_ok()
        for n, x in zip(("dq", "dk", "dv"), g):
            _within(x, r[n], r["tol_" + n], n)
    return r


SCORES = [
    # cap, slopes?, q multiplier: every range of the cap's approximations
    (0.0, False, 1.0), (50.0, False, 1.0), (12.0, False, 1.0), (4.0, False, 1.0), (1.0, False, 1.0),
    (50.0, False, 8.0), (0.0, True, 1.0), (50.0, True, 1.0), (3.0, True, 2.0),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", SCORES)
def test_scores_causal_without_a_plan(score, d):
    cap, bias, mult = score
    _run(1, 4, 2, 300, 300, d, True, cap, _slopes(4) if bias else None, mult=mult, planned=False)


SHAPES = [
    # B, Hq, Hkv, Sq, Sk, d, causal: one token to several tiles, heads in pairs and odd groups, Sq != Sk
    (1, 1, 1, 1, 1, 64, True), (2, 2, 1, 1, 130, 128, False), (1, 3, 3, 129, 127, 64, True),
    (1, 2, 2, 200, 700, 128, True), (2, 6, 2, 257, 257, 64, False), (1, 3, 1, 513, 400, 128, True),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score", [(0.0, False), (20.0, False), (0.0, True), (6.0, True)])
def test_shapes(shape, score):
    B, Hq, Hkv, Sq, Sk, d, causal = shape
    _run(B, Hq, Hkv, Sq, Sk, d, causal, score[0], _slopes(Hq) if score[1] else None, planned=False, seed=7)


MASKS = [
    # B, Sq, Sk, causal, window, cu, prefix
    (2, 300, 300, True, 0, [0, 1, 130, 300, 300, 520, 600], None),          # documents, a short one, an empty one
    (2, 300, 300, True, 0, [0, 100, 260, 300, 570, 600], [7, 130, -1, 0, -1]),  # prefixes and padding
    (2, 257, 257, False, 40, [0, 150, 257, 300, 514], None),               # documents seen both ways, a window
    (1, 400, 400, True, 1, None, None),                                    # every row sees itself
    (3, 140, 390, True, 64, None, [0, 200, 390]),                          # a chunk behind a prefix
    (1, 260, 260, True, 0, [30, 40, 200], None),                           # positions of no document
    (2, 130, 130, True, 0, None, [-1, 5]),                                 # a whole batch row of padding
    (1, 512, 512, True, 100, [0, 512], [300]),                             # a window inside a prefix
]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("score", [(0.0, False, 64), (30.0, False, 128), (0.0, True, 128), (5.0, True, 64)])
def test_masks(mask, score):
    B, Sq, Sk, causal, window, cu, prefix = mask
    cap, bias, d = score
    for Hq, Hkv in ((2, 1), (3, 3)):
        _run(B, Hq, Hkv, Sq, Sk, d, causal, cap, _slopes(Hq) if bias else None, window, cu, prefix, seed=11)


@pytest.mark.parametrize("Hq,Hkv,d,cap,bias", [(1, 1, 64, 0.0, False), (3, 3, 128, 9.0, True), (4, 2, 64, 9.0, False)])
@pytest.mark.parametrize("causal", [False, True])
def test_intervals_that_differ_from_tile_to_tile(causal, Hq, Hkv, d, cap, bias):
    # the caller's own intervals, one for each 128 rows: far apart within a pair of tiles, in both orders, one or
    # both without keys, an edge inside a tile; with the causal rule of the call on top
    B, S = 2, 900
    tiles = [[(0, 100), (700, 900), (700, 900), (0, 100), (0, 0), (128, 256), (5, 6), (9, 3)],
             [(0, 0), (5, 5), (0, 900), (899, 900), (127, 129), (255, 257), (300, 300), (0, 1)]]
    lo, hi = np.zeros((B, S), np.int64), np.zeros((B, S), np.int64)
    for b in range(B):
        for i in range(S):
            lo[b, i], hi[b, i] = tiles[b][i // 128]
    lo[1, 300], hi[1, 300] = -50, 5000  # clamped
    t = workloads.random_qkv(B, Hq, Hkv, S, S, d, seed=21, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    plan = fa.fa_mask_plan(_i32(lo.tolist()), _i32(hi.tolist()), S)
    sl = _slopes(Hq, 0.1) if bias else None
    how = dict(softcap=cap, slopes=None if sl is None else sl.to(DEV), plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, causal, 0.1, **how)
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, causal, 0.1, **how)
    torch.cuda.synchronize()
    _status_ok()
    lo, hi = np.maximum(lo, 0), np.minimum(hi, S)
    if causal:
        hi = np.minimum(hi, np.arange(S) + 1)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.1, lo, hi, cap, None if sl is None else sl.double().numpy(),
                  to_np(t["dout"]), bounds=True)
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    for n, x in zip(("dq", "dk", "dv"), g):
        _within(x, r[n], r["tol_" + n], n)


SPLIT = [
    # B, Hq, Hkv, Sq, Sk, d, causal, cap, slopes?, window, cu, prefix: few rows, keys of many tiles
    (1, 2, 1, 1, 2000, 64, True, 0.0, False, 0, None, None),
    (1, 3, 3, 130, 1700, 128, True, 20.0, True, 0, None, None),
    (2, 4, 2, 200, 2500, 64, False, 4.0, False, 0, None, None),
    (2, 2, 2, 300, 2000, 64, True, 0.0, True, 900, [0, 1850, 1900, 2000, 3000, 3990], [0, 0, 30, 1000, -1]),
    (1, 1, 1, 700, 1500, 128, True, 2.0, False, 0, [100, 1400], [1290]),
]


@pytest.mark.parametrize("case", SPLIT)
def test_few_rows_with_long_keys(case):
    # split over the GPU (with a workspace), the same without
    B, Hq, Hkv, Sq, Sk, d, causal, cap, bias, window, cu, prefix = case
    assert fa.fa_fwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) > 0
    sl = _slopes(Hq, 0.2) if bias else None
    planned = bool(window or cu)
    r = _run(B, Hq, Hkv, Sq, Sk, d, causal, cap, sl, window, cu, prefix, seed=31, planned=planned)
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=31, q_mult=1.0, with_dout=True)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    plan = None
    if planned:
        lo, hi = fa.fa_row_bounds(B, Sq, Sk, causal, window=window, cu_docs=_i32(cu), prefix=_i32(prefix))
        plan = fa.fa_mask_plan(lo, hi, Sk)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, Sq, device=DEV)
    slopes = None if sl is None else sl.to(DEV)
    st = fa.load_library().fa_fwd_scored(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Sk, d,
        int(causal and not planned), 1.0 / math.sqrt(d), cap, None if slopes is None else slopes.data_ptr(),
        None if plan is None else plan.data_ptr(), 0 if plan is None else plan.nbytes, None, 0, None)
    torch.cuda.synchronize()
    assert st == fa.FA_OK
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (9.0, False), (0.0, True), (3.0, True)])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,causal,window,cu,prefix", [
    (1, 16, 1, 400, 300, True, 0, None, None),                                # Sq > Sk: rows in front of the first key
    (1, 40, 2, 257, 130, False, 0, None, None),
    (2, 12, 1, 513, 513, True, 200, [0, 100, 260, 513, 800, 1026], [7, 0, -1, 300, 0]),
])
def test_backward_of_many_heads_on_few_keys(B, Hq, Hkv, Sq, Sk, causal, window, cu, prefix, cap, bias, d):
    # query heads and tiles of a key tile are split over the GPU
    assert fa.fa_bwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d) > fa.fa_bwd_workspace_size(B, Hq, Sq, d)
    _run(B, Hq, Hkv, Sq, Sk, d, causal, cap, _slopes(Hq, 0.3) if bias else None, window, cu, prefix, seed=41,
         planned=cu is not None)


def test_backward_of_many_heads_on_few_keys_where_nothing_looks():
    B, Hq, Hkv, S, d = 1, 24, 2, 420, 64
    cu, prefix = [0, 50, 370, 420], [-1, 0, -1]
    t = workloads.random_qkv(B, Hq, Hkv, S, S, d, seed=42, with_dout=True)
    lo, hi = so.row_bounds(B, S, S, True, 0, cu, prefix)
    dead = torch.from_numpy(hi <= lo)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.09, lo, hi, 9.0, None, to_np(t["dout"]), bounds=True)
    for x in t.values():
        x.masked_fill_(dead[:, None, :, None], float("nan"))
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    plan = fa.fa_mask_plan(*fa.fa_row_bounds(B, S, S, True, cu_docs=_i32(cu), prefix=_i32(prefix)), S)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.09, softcap=9.0, plan=plan)
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.09, softcap=9.0, plan=plan)
    torch.cuda.synchronize()
    _status_ok()
    for n, x in zip(("dq", "dk", "dv"), g):
        _within(x, r[n], r["tol_" + n], n)


def test_few_rows_with_long_keys_and_nan():
    # a NaN in a key or value reaches the rows that see it through the join as well; what lies in front of the first
    # and behind the last visible key is not used
    B, H, Sq, Sk, d = 1, 2, 100, 3000, 64
    t = workloads.random_qkv(B, H, H, Sq, Sk, d, seed=32)
    lo = np.full((B, Sq), 500)
    hi = np.full((B, Sq), 2600)
    hi[:, :10], hi[:, 10:20] = 2000, 0
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.1, lo, hi, 5.0, bounds=True)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    for x in (k, v):
        x[:, :, :500] = float("nan")
        x[:, :, 2600:] = float("inf")
    plan = fa.fa_mask_plan(_i32(lo.tolist()), _i32(hi.tolist()), Sk)
    assert fa.fa_fwd_scored_workspace_size(B, H, H, Sq, Sk, d) > 0
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=5.0, plan=plan)
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    k[:, :, 2400] = float("nan")
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=5.0, plan=plan)
    assert bool(o[:, :, 20:].isnan().all()) and bool(lse[:, :, 20:].isnan().all())
    assert bool((o[:, :, 10:20] == 0).all()) and bool((lse[:, :, 10:20] == -math.inf).all())
    _within(lse[:, :, :10], r["lse"][:, :, :10], r["tol_lse"][:, :, :10], "LSE")
    _status_ok()


def test_batch_rows_of_very_different_work_in_one_plan():
    # tiles go by their work over all batch rows together: each batch row as if it were alone
    B, S, H, d = 40, 384, 2, 64
    rng = np.random.RandomState(4)
    lo = np.sort(rng.randint(0, S, (B, S)), axis=1) * (rng.rand(B, 1) < 0.5)
    hi = np.minimum(S, lo + rng.randint(0, S, (B, 1)))
    t = workloads.random_qkv(B, H, H, S, S, d, seed=22, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    lo, hi = _i32(lo.tolist()), _i32(hi.tolist())
    plan = fa.fa_mask_plan(lo, hi, S)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.125, softcap=8.0, plan=plan)
    dq, dk, dv = fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.125, softcap=8.0, plan=plan)
    for b in range(0, B, 3):
        one = [x[b:b + 1].contiguous() for x in (q, k, v)]
        p1 = fa.fa_mask_plan(lo[b:b + 1].contiguous(), hi[b:b + 1].contiguous(), S)
        o1, l1 = fa.fa_fwd_scored(*one, False, 0.125, softcap=8.0, plan=p1)
        g1 = fa.fa_bwd_scored(*one, o1, do[b:b + 1].contiguous(), l1, False, 0.125, softcap=8.0, plan=p1)
        assert torch.equal(o[b], o1[0]) and torch.equal(lse[b], l1[0])
        assert torch.equal(dk[b], g1[1][0]) and torch.equal(dv[b], g1[2][0])
        # dQ is added in any order: fp32 sums of at most 3 tiles, then one rounding to bf16
        assert ((dq[b].float() - g1[0][0].float()).abs() <= 2.0 ** -7 * dq[b].float().abs() + 1e-6).all()
    _status_ok()


def test_steep_and_negative_slopes_and_scale_zero():
    steep = torch.tensor([40.0, -0.05, 0.0, 1e-4])
    _run(1, 4, 4, 300, 300, 128, True, 0.0, steep, planned=False)
    _run(1, 4, 2, 200, 300, 64, False, 9.0, steep, planned=False)
    _run(1, 4, 2, 200, 300, 64, True, 9.0, None, planned=False, scale=0.0)
    _run(1, 4, 2, 200, 300, 64, True, 0.0, steep, planned=False, scale=0.0)


def test_extreme_caps():
    # the folded coefficients do not fit fp32 here: tanh by special functions throughout
    for cap, scale in ((2.0 ** 20, 0.1), (2.0 ** -20, 0.1), (1.0, 300.0)):
        _run(1, 2, 1, 150, 150, 64, True, cap, None, planned=False, scale=scale, back=cap < 2.0 ** 20)


def test_callers_own_intervals():
    # intervals in no order at all, out of range, empty and inverted ones
    B, S, d = 2, 300, 64
    rng = np.random.RandomState(2)
    lo, hi = rng.randint(-50, S, (B, S)), rng.randint(0, S + 50, (B, S))
    lo[:, 5:9], hi[:, 5:9] = 200, 100
    t = workloads.random_qkv(B, 2, 2, S, S, d, seed=3, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    plan = fa.fa_mask_plan(_i32(lo), _i32(hi), S)
    for causal in (False, True):
        o, lse = fa.fa_fwd_scored(q, k, v, causal, 0.125, softcap=8.0, plan=plan)
        g = fa.fa_bwd_scored(q, k, v, o, do, lse, causal, 0.125, softcap=8.0, plan=plan)
        h = np.minimum(hi, np.arange(S) + 1) if causal else hi
        r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.125, np.maximum(lo, 0), np.minimum(h, S), 8.0, None,
                      to_np(t["dout"]), bounds=True)
        torch.cuda.synchronize()
        _status_ok()
        _within(o, r["o"], r["tol_o"], "O")
        _within(lse, r["lse"], r["tol_lse"], "LSE")
        for n, x in zip(("dq", "dk", "dv"), g):
            _within(x, r[n], r["tol_" + n], n)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (4.0, True)])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
def test_what_nothing_sees_may_hold_anything(garbage, cap, bias):
    # padding at both ends of a row: queries, keys, values and dO there are not used
    B, H, S, d = 2, 3, 420, 128
    cu, prefix = [0, 50, 370, 420, 520, 840], [-1, 0, -1, -1, 20]
    t = workloads.random_qkv(B, H, H, S, S, d, seed=5, with_dout=True)
    lo, hi = so.row_bounds(B, S, S, True, 0, cu, prefix)
    sl = _slopes(H) if bias else None
    dead = torch.from_numpy(hi <= lo)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.09, lo, hi, cap, None if sl is None else sl.double().numpy(),
                  to_np(t["dout"]), bounds=True)
    for x in t.values():
        x.masked_fill_(dead[:, None, :, None], garbage)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    plan = fa.fa_mask_plan(*fa.fa_row_bounds(B, S, S, True, cu_docs=_i32(cu), prefix=_i32(prefix)), S)
    how = dict(softcap=cap, slopes=None if sl is None else sl.to(DEV), plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.09, **how)
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.09, **how)
    torch.cuda.synchronize()
    _status_ok()
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse, r["lse"], r["tol_lse"], "LSE")
    for n, x in zip(("dq", "dk", "dv"), g):
        _within(x, r[n], r["tol_" + n], n)
        assert float(x.masked_select(dead[:, None, :, None].to(DEV)).abs().sum()) == 0.0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias,planned", [(0.0, False, False), (0.0, False, True), (20.0, False, True),
                                              (0.0, True, False), (2.0, True, True)])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_a_nan_reaches_the_rows_that_see_it(where, cap, bias, planned, d):
    # and none outside of their 256-row blocks: row 300 (of q), or key 300 (of k or v) under the causal rule
    B, H, S, at = 1, 2, 700, 300
    t = workloads.random_qkv(B, H, H, S, S, d, seed=5, with_dout=True)
    sl = _slopes(H) if bias else None
    lo, hi = so.row_bounds(B, S, S, True)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.09, lo, hi, cap, None if sl is None else sl.double().numpy(),
                  to_np(t["dout"]), bounds=True)
    t[where][:, :, at] = float("nan")
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    plan = fa.fa_mask_plan(*fa.fa_row_bounds(B, S, S, True), S) if planned else None
    how = dict(softcap=cap, slopes=None if sl is None else sl.to(DEV), plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, not planned, 0.09, **how)
    dq, dk, dv = fa.fa_bwd_scored(q, k, v, o, do, lse, not planned, 0.09, **how)
    torch.cuda.synchronize()
    _status_ok()
    sees = slice(at, at + 1) if where == "q" else slice(at, S)
    assert bool(o[:, :, sees].isnan().all())
    assert bool(dq[:, :, sees].isnan().all())
    if where != "v":
        assert bool(lse[:, :, sees].isnan().all())
        assert bool(dk[:, :, :at + 1].isnan().all())
    else:
        _within(lse, r["lse"], r["tol_lse"], "LSE")
    for part in [slice(0, 256)] + ([slice(512, S)] if where == "q" else []):
        _within(o[:, :, part], r["o"][:, :, part], r["tol_o"][:, :, part], "O")
        _within(dq[:, :, part], r["dq"][:, :, part], r["tol_dq"][:, :, part], "dq")
        _within(lse[:, :, part], r["lse"][:, :, part], r["tol_lse"][:, :, part], "LSE")


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_decode_a_nan_reaches_the_rows_that_see_it(cap, Hq, Hkv, d):
    lens, room, at = [700, 300, 301, 699, 1], 700, 300
    B = len(lens)
    t = workloads.random_qkv(B, Hq, Hkv, 1, room, d, seed=6)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    for where in (k, v):
        clean = fa.fa_decode_scored(q, k, v, _i32(lens), 0.1, cap), fa.fa_decode_scored(q, k, v, _i32(lens), 0.1, cap, window=390)
        kept = where[:, :, at].clone()
        where[:, :, at] = float("nan")
        dirty = fa.fa_decode_scored(q, k, v, _i32(lens), 0.1, cap), fa.fa_decode_scored(q, k, v, _i32(lens), 0.1, cap, window=390)
        where[:, :, at] = kept
        for (o0, l0), (o, lse), windowed in zip(clean, dirty, (False, True)):
            for b, n in enumerate(lens):
                if n > at and not (windowed and n - 390 > at):
                    assert bool(o[b].isnan().all()), (n, windowed)
                    assert bool(lse[b].isnan().all()) == (where is k), (n, windowed)
                else:
                    assert torch.equal(o[b], o0[b]) and torch.equal(lse[b], l0[b]), (n, windowed)
    _status_ok()


def test_plain_scores_equal_the_plain_kernels():
    # without cap, bias and plan these are fa_fwd's sums over the same tiles: equal up to the order of tiles
    t = workloads.random_qkv(2, 4, 2, 300, 300, 128, seed=9)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    o0, l0 = fa.fa_fwd(q, k, v, True, 0.09)
    o1, l1 = fa.fa_fwd_scored(q, k, v, True, 0.09)
    assert (o0.float() - o1.float()).abs().max() <= 2 * 2.0 ** -8 * v.float().abs().max()
    assert (l0 - l1).abs().max() <= 1e-5


def test_many_units_per_block_and_their_order():
    # more units than SMs, of very different work, against the same documents one call at a time
    S, H, d = 1024, 8, 64
    rng = np.random.RandomState(6)
    B = 5
    cuts = np.sort(rng.randint(0, B * S, 14))
    cu = [0] + [int(c) for c in cuts] + [B * S]
    t = workloads.random_qkv(B, H, 4, S, S, d, seed=10, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    lo, hi = fa.fa_row_bounds(B, S, S, True, cu_docs=_i32(cu))
    plan = fa.fa_mask_plan(lo, hi, S)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.125, softcap=10.0, plan=plan)
    g = fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.125, softcap=10.0, plan=plan)
    for b in range(B):
        pl = fa.fa_mask_plan(lo[b:b + 1].contiguous(), hi[b:b + 1].contiguous(), S)
        x = [y[b:b + 1].contiguous() for y in (q, k, v, do)]
        ob, lb = fa.fa_fwd_scored(*x[:3], False, 0.125, softcap=10.0, plan=pl)
        gb = fa.fa_bwd_scored(*x[:3], ob, x[3], lb, False, 0.125, softcap=10.0, plan=pl)
        assert torch.equal(ob[0], o[b]) and torch.equal(lb[0], lse[b])
        assert torch.equal(gb[1][0], g[1][b]) and torch.equal(gb[2][0], g[2][b])
        # dQ's partial sums are added in the order the tiles finish: fp32 before the rounding to bf16
        assert (gb[0][0].float() - g[0][b].float()).abs().max() <= 2.0 ** -8 * g[0][b].float().abs().max()
    _status_ok()


# ------------------------------------------------------------------- masks --

@pytest.mark.parametrize("causal", [False, True])
def test_row_bounds_of_many_documents(causal):
    rng = np.random.RandomState(1)
    for B, Sq, Sk, n, window in ((3, 50, 50, 9, 0), (2, 33, 70, 5, 12), (1, 500, 500, 200, 3), (4, 7, 7, 1, 0)):
        cu = np.sort(rng.randint(0, B * Sk + 1, n + 1)).tolist()
        pre = rng.randint(-1, 20, n).tolist()
        for p in (None, pre):
            lo, hi = fa.fa_row_bounds(B, Sq, Sk, causal, window=window, cu_docs=_i32(cu), prefix=_i32(p))
            wl, wh = so.row_bounds(B, Sq, Sk, causal, window, cu, p)
            assert np.array_equal(lo.cpu().numpy(), wl) and np.array_equal(hi.cpu().numpy(), wh)
    lo, hi = fa.fa_row_bounds(2, 5, 9, causal, window=3, prefix=_i32([4, -1]))
    wl, wh = so.row_bounds(2, 5, 9, causal, 3, None, [4, -1])
    assert np.array_equal(lo.cpu().numpy(), wl) and np.array_equal(hi.cpu().numpy(), wh)


def test_row_bounds_past_32_bit_products():
    # the flattened positions reach 2^31 - 128; a document's far end and prefix near the largest int
    B, S = 1, (1 << 31) - 128
    lo, hi = fa.fa_row_bounds(B, 4, S, True, cu_docs=_i32([0, S - 2, S]), prefix=_i32([2 ** 31 - 1, 2 ** 31 - 1]))
    assert lo.tolist() == [[0, 0, S - 2, S - 2]] and hi.tolist() == [[S - 2, S - 2, S, S]]
    lo, hi = fa.fa_row_bounds(B, 4, S, False, window=2 ** 31 - 1)
    assert lo.tolist() == [[0] * 4] and hi.tolist() == [[S] * 4]


# ------------------------------------------------------------------ decode --

DECODE = [
    # B, Hq, Hkv, d, Sk_max, lens, window, starts, cap, bias
    (1, 1, 1, 64, 1, [1], 0, None, 0.0, False),
    (3, 8, 2, 128, 1500, [1500, 1, 777], 0, None, 50.0, False),
    (4, 6, 2, 64, 900, [0, 900, 130, 899], 100, None, 0.0, True),
    (4, 16, 1, 128, 700, [700, 64, 5, 300], 0, [0, 64, 3, 299], 6.0, True),
    (2, 24, 2, 64, 2000, [2000, 1999], 513, [1900, 0], 2.0, False),
    (2, 4, 4, 128, 9000, [9000, 4321], 4096, None, 30.0, True),
    (3, 2, 2, 64, 300, [400, -5, 300], 0, [-7, 0, 1000], 10.0, False),   # clamped lengths and starts
    # short items, each one block's
    (12, 12, 4, 128, 1024, [1024, 0, 1, 127, 128, 129, 1023, 500, 384, 2, 0, 700], 0, None, 8.0, True),
    (12, 12, 4, 128, 1024, [1024, 0, 1, 127, 128, 129, 1023, 500, 384, 2, 0, 700], 300, [0, 0, 1, 120] + [3] * 8, 0.0, True),
    (5, 40, 2, 64, 500, [500, 256, 257, 0, 77], 0, [499, 0, 256, 0, 80], 3.0, True),
    (19, 16, 16, 64, 1500, [79 * i for i in range(19)], 0, None, 20.0, False),
    (3, 8, 8, 128, 5000, [5000, 130, 4099], 200, None, 2.0, True),
]


@pytest.mark.parametrize("case", DECODE)
def test_decode(case):
    B, Hq, Hkv, d, Sk, lens, window, starts, cap, bias = case
    t = workloads.random_qkv(B, Hq, Hkv, 1, Sk, d, seed=13, q_mult=2.0)
    sl = _slopes(Hq) if bias else None
    n = np.clip(lens, 0, Sk)
    lo = np.maximum(0, np.array(starts)) if starts else np.zeros(B, np.int64)
    if window:
        lo = np.maximum(lo, n - window)
    # what lies outside of the interval is never read
    for b in range(B):
        for x in (t["k"], t["v"]):
            x[b, :, n[b]:] = float("nan")
            x[b, :, :min(lo[b], n[b])] = float("nan")
    o, lse = fa.fa_decode_scored(t["q"].to(DEV), t["k"].to(DEV), t["v"].to(DEV), _i32(lens), 0.11, softcap=cap,
                                 slopes=None if sl is None else sl.to(DEV), window=window, k_start=_i32(starts))
    torch.cuda.synchronize()
    _status_ok()
    for b in range(B):
        # as a row at the last of n positions
        m = max(1, int(n[b]))
        kk, vv = (torch.nan_to_num(t[x][b:b + 1, :, :m]).double().numpy() for x in ("k", "v"))
        r = so.attend(to_np(t["q"][b:b + 1]), kk, vv, 0.11, np.array([[lo[b]]]), np.array([[n[b]]]), cap,
                      None if sl is None else sl.double().numpy(), bounds=True)
        _within(o[b:b + 1], r["o"], r["tol_o"], f"O {b}")
        _within(lse[b:b + 1, :, None], r["lse"], r["tol_lse"], f"LSE {b}")


def test_decode_equals_the_last_row_of_the_forward():
    B, Hq, Hkv, S, d = 2, 8, 4, 333, 128
    t = workloads.random_qkv(B, Hq, Hkv, 1, S, d, seed=14, q_mult=3.0)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    sl = _slopes(Hq).to(DEV)
    lo, hi = fa.fa_row_bounds(B, 1, S, True, window=200)
    o0, l0 = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=15.0, slopes=sl, plan=fa.fa_mask_plan(lo, hi, S))
    o1, l1 = fa.fa_decode_scored(q, k, v, _i32([S, S]), 0.1, softcap=15.0, slopes=sl, window=200)
    # the forward rounds weights to bf16, the decode does not
    assert (o0.float() - o1.float()).abs().max() <= 3 * 2.0 ** -8 * v.float().abs().max()
    assert (l0[..., 0] - l1).abs().max() <= 1e-4


# ------------------------------------------------- streams, graphs, outputs --

def test_other_stream_and_given_outputs():
    t = workloads.random_qkv(1, 2, 1, 200, 200, 64, seed=15, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    lo, hi = fa.fa_row_bounds(1, 200, 200, True, window=50)
    plan = fa.fa_mask_plan(lo, hi, 200)
    o0, l0 = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=5.0, plan=plan)
    g0 = fa.fa_bwd_scored(q, k, v, o0, do, l0, False, 0.1, softcap=5.0, plan=plan)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [torch.full_like(x, 7.0) for x in (o0, l0, *g0)]
    ws = torch.empty(fa.fa_bwd_workspace_size(1, 2, 200, 64), dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    lo1, hi1 = fa.fa_row_bounds(1, 200, 200, True, window=50, stream=s)
    plan1 = fa.fa_mask_plan(lo1, hi1, 200, stream=s)
    o1, l1 = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=5.0, plan=plan1, o=outs[0], lse=outs[1], stream=s)
    fa.fa_bwd_scored(q, k, v, o1, do, l1, False, 0.1, softcap=5.0, plan=plan1, dq=outs[2], dk=outs[3], dv=outs[4],
                     workspace=ws, stream=s)
    s.synchronize()
    _status_ok()
    assert o1 is outs[0] and torch.equal(o0, outs[0]) and torch.equal(l0, outs[1])
    assert torch.equal(g0[1], outs[3]) and torch.equal(g0[2], outs[4])
    assert (g0[0].float() - outs[2].float()).abs().max() <= 2.0 ** -8 * g0[0].float().abs().max()


def test_captured_step_follows_new_inputs():
    # masks, forward, backward and a decode in one graph; replayed with other inputs and other documents
    B, H, S, d = 2, 2, 256, 64
    shapes = dict(q=(B, H, S, d), k=(B, H, S, d), v=(B, H, S, d), dout=(B, H, S, d))
    buf = {n: torch.zeros(s, dtype=BF, device=DEV) for n, s in shapes.items()}
    cu = _i32([0, S, 2 * S])
    lens = _i32([S, S])
    sl = _slopes(H).to(DEV)

    def step():
        lo, hi = fa.fa_row_bounds(B, S, S, True, window=100, cu_docs=cu)
        plan = fa.fa_mask_plan(lo, hi, S)
        how = dict(softcap=6.0, slopes=sl, plan=plan)
        o, lse = fa.fa_fwd_scored(buf["q"], buf["k"], buf["v"], False, 0.125, **how)
        g = fa.fa_bwd_scored(buf["q"], buf["k"], buf["v"], o, buf["dout"], lse, False, 0.125, **how)
        od, _ = fa.fa_decode_scored(buf["q"][:, :, -1:].contiguous(), buf["k"], buf["v"], lens, 0.125, softcap=6.0,
                                    slopes=sl, window=64)
        return (o, lse, *g, od)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed, docs, ln in ((1, [0, S, 2 * S], [S, S]), (2, [0, 100, 300], [17, 200])):
        for n, x in workloads.random_qkv(B, H, H, S, S, d, seed=seed, with_dout=True).items():
            buf[n].copy_(x)
        cu.copy_(_i32(docs))
        lens.copy_(_i32(ln))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        want = step()
        torch.cuda.synchronize()
        _status_ok()
        for i, (a, b) in enumerate(zip(got, want)):
            if i == 2:  # dQ: order of additions
                assert (a.float() - b.float()).abs().max() <= 2.0 ** -8 * b.float().abs().max()
            else:
                assert torch.equal(a, b), i


def test_binding_checks_shapes_and_devices():
    q = torch.zeros(1, 2, 8, 64, dtype=BF, device=DEV)
    k = torch.zeros(1, 1, 9, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q, k, q, True, 0.1)
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q, k, k, True, 0.1, slopes=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, True, 0.1)
    with pytest.raises(ValueError):  # the plan of other sizes
        fa.fa_fwd_scored(q, k, k, True, 0.1, plan=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(fa.FAError):
        fa.fa_fwd_scored(q, k, k, True, 0.1, softcap=-1.0)
    with pytest.raises(fa.FAError):
        fa.fa_decode_scored(q[:, :, :1].contiguous(), k, k, _i32([9]), 0.1, window=-1)
    with pytest.raises(ValueError):
        fa.fa_row_bounds(2, 8, 8, True, prefix=_i32([1]))
