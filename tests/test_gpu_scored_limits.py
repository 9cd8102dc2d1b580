"""The operators around the scores at their limits: stray writes (outputs and workspaces carved out of sentinel-filled
buffers), offsets past 32 bits, long sequences, many requests, and heads in numbers that fill no tile."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads
from oracle import scored as so
from tests.parity import to_np
from tests.test_gpu_guard import SENT, Carved
from tests.test_gpu_scored import _i32, _slopes, _status_ok, _within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _carve(*shapes):
    return [Carved(s, t) for s, t in shapes]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (3, 3)])
def test_attention_writes_its_outputs_and_nothing_else(d, Hq, Hkv):
    B, Sq, Sk = 2, 129, 300
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=1, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    cu = _i32([0, 250, 300, 400, 590])
    lo, hi, plan, o, lse, dq, dk, dv, ws = _carve(
        ((B, Sq), torch.int32), ((B, Sq), torch.int32), ((fa.fa_mask_plan_size(B, Sq, Sk),), torch.uint8),
        ((B, Hq, Sq, d), BF), ((B, Hq, Sq), torch.float32), ((B, Hq, Sq, d), BF), ((B, Hkv, Sk, d), BF),
        ((B, Hkv, Sk, d), BF), ((fa.fa_bwd_workspace_size(B, Hq, Sq, d),), torch.uint8))
    fa.fa_row_bounds(B, Sq, Sk, True, window=90, cu_docs=cu, row_lo=lo.t, row_hi=hi.t)
    fa.fa_mask_plan(lo.t, hi.t, Sk, plan=plan.t)
    how = dict(softcap=9.0, slopes=_slopes(Hq).to(DEV), plan=plan.t)
    fa.fa_fwd_scored(q, k, v, False, 0.1, o=o.t, lse=lse.t, **how)
    fa.fa_bwd_scored(q, k, v, o.t, do, lse.t, False, 0.1, dq=dq.t, dk=dk.t, dv=dv.t, workspace=ws.t, **how)
    torch.cuda.synchronize()
    _status_ok()
    for n, c in dict(lo=lo, hi=hi, plan=plan, o=o, lse=lse, dq=dq, dk=dk, dv=dv, workspace=ws).items():
        c.check_guards(n)
    for n, c in dict(o=o, dq=dq, dk=dk, dv=dv).items():
        assert not c.untouched_rows(np.zeros(c.t.numel() // d)).any(), n


def test_split_backward_writes_its_outputs_and_nothing_else():
    B, Hq, Hkv, Sq, Sk, d = 1, 24, 1, 140, 300, 64
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=5, with_dout=True)
    nbytes = fa.fa_bwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d)
    assert nbytes > fa.fa_bwd_workspace_size(B, Hq, Sq, d)
    dq, dk, dv, ws = _carve(((B, Hq, Sq, d), BF), ((B, Hkv, Sk, d), BF), ((B, Hkv, Sk, d), BF), ((nbytes,), torch.uint8))
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    o, lse = fa.fa_fwd_scored(q, k, v, True, 0.1, softcap=6.0)
    lo, hi = so.row_bounds(B, Sq, Sk, True)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.1, lo, hi, 6.0, None, to_np(t["dout"]), bounds=True)
    first = None
    for _ in range(2):
        ws.t.fill_(0xff)  # every part is written anew
        fa.fa_bwd_scored(q, k, v, o, do, lse, True, 0.1, softcap=6.0, dq=dq.t, dk=dk.t, dv=dv.t, workspace=ws.t)
        torch.cuda.synchronize()
        _status_ok()
        for n, c in dict(dq=dq, dk=dk, dv=dv, workspace=ws).items():
            c.check_guards(n)
        for n, c in dict(dq=dq, dk=dk, dv=dv).items():
            _within(c.t, r[n], r["tol_" + n], n)
        if first:  # parts are added in order
            assert torch.equal(first[0], dk.t) and torch.equal(first[1], dv.t)
        first = dk.t.clone(), dv.t.clone()


def test_split_attention_writes_its_outputs_and_nothing_else():
    B, Hq, Hkv, Sq, Sk, d = 1, 3, 1, 70, 2100, 64
    t = workloads.random_qkv(B, Hq, Hkv, Sq, Sk, d, seed=4)
    nbytes = fa.fa_fwd_scored_workspace_size(B, Hq, Hkv, Sq, Sk, d)
    assert nbytes > 0
    o, lse, ws = _carve(((B, Hq, Sq, d), BF), ((B, Hq, Sq), torch.float32), ((nbytes,), torch.uint8))
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    fa.fa_fwd_scored(q, k, v, True, 0.1, softcap=6.0, o=o.t, lse=lse.t, workspace=ws.t)
    # captured and replayed over the same workspace
    g = torch.cuda.CUDAGraph()
    o2, lse2 = torch.empty_like(q), torch.empty(B, Hq, Sq, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        fa.fa_fwd_scored(q, k, v, True, 0.1, softcap=6.0, o=o2, lse=lse2, workspace=ws.t)
    ws.t.fill_(0xff)  # every part is written anew
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    _status_ok()
    for n, c in dict(o=o, lse=lse, workspace=ws).items():
        c.check_guards(n)
    assert torch.equal(o.t, o2) and torch.equal(lse.t, lse2)
    lo, hi = so.row_bounds(B, Sq, Sk, True)
    r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 0.1, lo, hi, 6.0, bounds=True)
    _within(o2, r["o"], r["tol_o"], "O")
    _within(lse2, r["lse"], r["tol_lse"], "LSE")


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (20, 1), (33, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_writes_its_outputs_and_nothing_else(Hq, Hkv, d):
    B, Sk = 3, 777
    t = workloads.random_qkv(B, Hq, Hkv, 1, Sk, d, seed=2)
    lens = [777, 0, 130]
    nbytes = fa.fa_decode_scored_workspace_size(B, Hq, Hkv, Sk, d, 0)
    o, lse, ws = _carve(((B, Hq, 1, d), BF), ((B, Hq), torch.float32), ((nbytes,), torch.uint8))
    fa.fa_decode_scored(t["q"].to(DEV), t["k"].to(DEV), t["v"].to(DEV), _i32(lens), 0.1, softcap=5.0, o=o.t, lse=lse.t,
                        workspace=ws.t)
    torch.cuda.synchronize()
    _status_ok()
    for n, c in dict(o=o, lse=lse, workspace=ws).items():
        c.check_guards(n)
    for b, n in enumerate(lens):
        m = max(1, n)
        r = so.attend(to_np(t["q"][b:b + 1]), to_np(t["k"][b:b + 1, :, :m]), to_np(t["v"][b:b + 1, :, :m]), 0.1,
                      np.array([[0]]), np.array([[n]]), 5.0, bounds=True)
        _within(o.t[b:b + 1], r["o"], r["tol_o"], f"O {b}")
        _within(lse.t[b:b + 1, :, None], r["lse"], r["tol_lse"], f"LSE {b}")


def test_prep_writes_its_outputs_and_nothing_else():
    B, S, Hq, Hkv, d = 2, 37, 5, 3, 64
    g = torch.Generator().manual_seed(4)
    rows = torch.randn(B, S, Hq + 2 * Hkv, d, generator=g).to(BF).to(DEV)
    x = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).to(DEV)
    f = torch.rand(16, generator=g).to(DEV)
    how = dict(inv_freq=f, q_weight=w, k_weight=w)
    heads = lambda h: ((B, h, S, d), BF)  # noqa: E731
    q, k, v = _carve(heads(Hq), heads(Hkv), heads(Hkv))
    fa.fa_qk_norm_rope(*x, **how, q_out=q.t, k_out=k.t, v_out=v.t)
    dq, dk, dv, dwq, dwk, ws = _carve(((B, S, Hq, d), BF), ((B, S, Hkv, d), BF), ((B, S, Hkv, d), BF),
                                      ((d,), torch.float32), ((d,), torch.float32),
                                      ((fa.fa_qk_norm_rope_bwd_workspace_size(d),), torch.uint8))
    fa.fa_qk_norm_rope_bwd(x[0], x[1], q.t, k.t, v.t, **how, dq=dq.t, dk=dk.t, dv=dv.t, dq_weight=dwq.t, dk_weight=dwk.t,
                           workspace=ws.t)
    torch.cuda.synchronize()
    for n, c in dict(q=q, k=k, v=v, dq=dq, dk=dk, dv=dv, dwq=dwq, dwk=dwk, workspace=ws).items():
        c.check_guards(n)
    for n, c in dict(q=q, k=k, v=v, dq=dq, dk=dk, dv=dv).items():
        assert not c.untouched_rows(np.zeros(c.t.numel() // d)).any(), n
    assert not bool((dwq.buf[8192:8192 + 4 * d] == SENT).all())
    # a gradient into the middle of a wider buffer leaves the rest of it
    wide = torch.full((B, S + 4, Hq + 2 * Hkv + 2, d + 32), 3.0, dtype=BF, device=DEV)
    view = wide[:, 2:S + 2, 1:Hq + 1, 8:d + 8]
    fa.fa_qk_norm_rope_bwd(x[0], x[1], q.t, k.t, **how, dq=view)
    assert torch.equal(view, dq.t)
    view.fill_(3.0)
    assert bool((wide == 3.0).all())


def test_long_sequence_with_window_and_documents():
    S, H, d, window = 131_072, 1, 64, 200
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v, do = (torch.randn(1, H, S, d, generator=g, device=DEV).to(BF) for _ in range(4))
    cu = [0, 1000, 70_001, S]
    lo, hi = fa.fa_row_bounds(1, S, S, True, window=window, cu_docs=_i32(cu))
    plan = fa.fa_mask_plan(lo, hi, S)
    sl = torch.tensor([0.01], device=DEV)
    how = dict(softcap=15.0, slopes=sl, plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.125, **how)
    dq, dk, dv = fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.125, **how)
    torch.cuda.synchronize()
    _status_ok()
    lo, hi = lo.cpu().numpy(), hi.cpu().numpy()
    for a, b in ((0, 600), (900, 1500), (69_800, 70_500), (S - 700, S)):
        # rows from a + window on see only keys of the slice; keys up to b - window are seen only by its rows
        cut = [to_np(x[:, :, a:b]) for x in (q, k, v, do)]
        r = so.attend(*cut[:3], 0.125, np.maximum(lo[:, a:b] - a, 0), np.maximum(hi[:, a:b] - a, 0), 15.0, [0.01], cut[3],
                      bounds=True)
        rows = slice(0 if a == 0 else window, b - a)
        keys = slice(0 if a == 0 else window, b - a if b == S else b - a - window)
        _within(o[:, :, a:b][:, :, rows], r["o"][:, :, rows], r["tol_o"][:, :, rows], "O")
        _within(lse[:, :, a:b][:, :, rows], r["lse"][:, :, rows], r["tol_lse"][:, :, rows], "LSE")
        _within(dq[:, :, a:b][:, :, rows], r["dq"][:, :, rows], r["tol_dq"][:, :, rows], "dQ")
        for n, x in (("dk", dk), ("dv", dv)):
            _within(x[:, :, a:b][:, :, keys], r[n][:, :, keys], r["tol_" + n][:, :, keys], n)


def test_decode_of_many_requests():
    # more batch rows than one pass over the lengths takes, most of them short or empty
    B, Hq, Hkv, Sk, d = 1000, 4, 2, 400, 64
    rng = np.random.RandomState(6)
    lens = np.where(rng.rand(B) < 0.4, 0, rng.randint(1, Sk + 1, B))
    g = torch.Generator(device=DEV).manual_seed(7)
    q = torch.randn(B, Hq, 1, d, generator=g, device=DEV).to(BF)
    k, v = (torch.randn(B, Hkv, Sk, d, generator=g, device=DEV).to(BF) for _ in range(2))
    starts = rng.randint(0, 200, B)
    o, lse = fa.fa_decode_scored(q, k, v, _i32(lens), 0.125, softcap=8.0, window=150, k_start=_i32(starts))
    torch.cuda.synchronize()
    _status_ok()
    first = np.maximum(starts, lens - 150)
    for b in list(rng.choice(B, 40, replace=False)) + [0, B - 1]:
        n = int(lens[b])
        if first[b] >= n:
            assert float(o[b].abs().sum()) == 0.0 and bool(torch.isinf(lse[b]).all())
            continue
        r = so.attend(to_np(q[b:b + 1]), to_np(k[b:b + 1, :, :n]), to_np(v[b:b + 1, :, :n]), 0.125,
                      np.array([[first[b]]]), np.array([[n]]), 8.0, bounds=True)
        _within(o[b:b + 1], r["o"], r["tol_o"], f"O {b}")
        _within(lse[b:b + 1, :, None], r["lse"], r["tol_lse"], f"LSE {b}")
    empty = torch.from_numpy(first >= lens).to(DEV)
    assert bool((o[empty] == 0).all()) and bool(torch.isinf(lse[empty]).all())


def test_decode_offsets_past_32_bits():
    # a cache of 2.4e9 elements: the last head's last keys lie past 2^31
    B, H, Sk, d = 1, 9, 2_100_000, 128
    k = torch.zeros(B, H, Sk, d, dtype=BF, device=DEV)
    v = torch.zeros(B, H, Sk, d, dtype=BF, device=DEV)
    n = Sk - 5
    g = torch.Generator(device=DEV).manual_seed(8)
    k[:, :, n - 300:n] = torch.randn(B, H, 300, d, generator=g, device=DEV).to(BF)
    v[:, :, n - 300:n] = torch.randn(B, H, 300, d, generator=g, device=DEV).to(BF)
    q = torch.randn(B, H, 1, d, generator=g, device=DEV).to(BF)
    o, lse = fa.fa_decode_scored(q, k, v, _i32([n]), 0.1, softcap=20.0, window=300)
    torch.cuda.synchronize()
    _status_ok()
    r = so.attend(to_np(q), to_np(k[:, :, n - 300:n]), to_np(v[:, :, n - 300:n]), 0.1, np.array([[0]]), np.array([[300]]),
                  20.0, bounds=True)
    _within(o, r["o"], r["tol_o"], "O")
    _within(lse[..., None], r["lse"], r["tol_lse"], "LSE")


def test_prep_offsets_past_32_bits():
    # 2.2e9 elements of projection rows; the last tokens against the same tokens alone
    B, S, Hq, Hkv, d = 1, 360_000, 32, 8, 128
    rows = torch.zeros(B, S, Hq + 2 * Hkv, d, dtype=BF, device=DEV)
    tail = torch.randn(B, 50, Hq + 2 * Hkv, d, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV).to(BF)
    rows[:, -50:] = tail
    f = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().to(DEV)
    w = torch.ones(d, dtype=BF, device=DEV)
    split = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])  # noqa: E731
    q, k, v = fa.fa_qk_norm_rope(*split(rows), inv_freq=f, q_weight=w, k_weight=w)
    pos = torch.arange(S - 50, S, dtype=torch.int32, device=DEV)[None]
    want = fa.fa_qk_norm_rope(*split(tail), positions=pos, inv_freq=f, q_weight=w, k_weight=w)
    for a, b in zip((q, k, v), want):
        assert torch.equal(a[:, :, -50:], b)
    del q, k, v
    gq, gk, gv = (torch.zeros(B, h, S, d, dtype=BF, device=DEV) for h in (Hq, Hkv, Hkv))
    for a, b in zip((gq, gk, gv), want):
        a[:, :, -50:] = b
    out = torch.empty_like(rows)
    fa.fa_qk_norm_rope_bwd(*split(rows)[:2], gq, gk, gv, inv_freq=f, q_weight=w, k_weight=w,
                           **dict(zip(("dq", "dk", "dv"), split(out))))
    small = fa.fa_qk_norm_rope_bwd(*split(tail)[:2], *want, positions=pos, inv_freq=f, q_weight=w, k_weight=w)
    for a, b in zip(split(out), small):
        assert torch.equal(a[:, -50:], b)


def test_scores_that_overflow_the_running_maximum_and_come_back():
    # scores that jump by hundreds between tiles, in both directions, without a cap
    B, H, S, d = 1, 2, 700, 64
    t = workloads.random_qkv(B, H, H, S, S, d, seed=12)
    jump = torch.ones(S)
    jump[:128], jump[256:384], jump[600:] = 30.0, 0.01, 60.0
    t["k"] = (t["k"].float() * jump[:, None]).to(BF)
    q, k, v = (t[n].to(DEV) for n in ("q", "k", "v"))
    lo, hi = so.row_bounds(B, S, S, False)
    for causal in (False, True):
        if causal:
            lo, hi = so.row_bounds(B, S, S, True)
        o, lse = fa.fa_fwd_scored(q, k, v, causal, 1.0 / math.sqrt(d))
        r = so.attend(*(to_np(t[n]) for n in ("q", "k", "v")), 1.0 / math.sqrt(d), lo, hi, bounds=True)
        torch.cuda.synchronize()
        _status_ok()
        _within(o, r["o"], r["tol_o"], "O")
        _within(lse, r["lse"], r["tol_lse"], "LSE")


@pytest.mark.parametrize("B,H,S,planned", [(2, 2, 65536, True), (8, 2, 16384, True), (2, 2, 65536, False)])
def test_backward_in_groups_that_fit_the_l2_cache(B, H, S, planned):
    # the gradients' accumulators exceed twice the L2: heads go group by group, in alternating order of work
    d = 128
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v, do = (torch.randn(B, H, S, d, device=DEV, dtype=BF, generator=g) for _ in range(4))
    if not planned:  # the causal rule alone, over fewer keys than queries, to keep it short
        k, v = k[:, :, :1024].contiguous(), v[:, :, :1024].contiguous()
    Sk = k.shape[2]
    cu = torch.arange(0, B * S + 1, 1000, dtype=torch.int32, device=DEV)
    cu[-1] = B * S

    def run(rows, heads):
        x = [y[rows, heads].contiguous() for y in (q, k, v, do)]
        plan = None
        if planned:
            plan = fa.fa_mask_plan(lo[rows].contiguous(), hi[rows].contiguous(), Sk)
        o, lse = fa.fa_fwd_scored(*x[:3], not planned, 0.09, softcap=20.0, plan=plan)
        # (with this workspace few keys are not split over the GPU, so that dK and dV are sums of one order)
        ws = torch.empty(fa.fa_bwd_workspace_size(*lse.shape[:2], S, d), dtype=torch.uint8, device=DEV)
        return (o, lse) + fa.fa_bwd_scored(*x[:3], o, x[3], lse, not planned, 0.09, softcap=20.0, plan=plan,
                                           workspace=ws)

    if planned:
        lo, hi = fa.fa_row_bounds(B, S, Sk, True, window=300, cu_docs=cu)
    every = run(slice(0, B), slice(0, H))
    for b in range(0, B, max(1, B - 1)):
        one = run(slice(b, b + 1), slice(H - 1, H))
        for n, x, y in zip(("o", "lse", "dq", "dk", "dv"), every, one):
            x = x[b:b + 1, H - 1:H]
            if n == "dq":  # added in any order: fp32 sums, then one rounding to bf16
                far = (x.float() - y.float()).abs() - 2.0 ** -7 * y.float().abs()
                assert float(far.max()) <= 1e-5 * float(y.float().abs().max())
            else:
                assert torch.equal(x, y), n
    _status_ok()


def test_two_steps_at_once_on_two_streams():
    # the same plan and caches read by two streams; outputs and workspaces of their own
    B, H, S, d = 2, 4, 512, 64
    t = [workloads.random_qkv(B, H, H, S, S, d, seed=s, with_dout=True) for s in (20, 21)]
    dev = [{n: x.to(DEV) for n, x in y.items()} for y in t]
    lo, hi = fa.fa_row_bounds(B, S, S, True, window=300)
    plan = fa.fa_mask_plan(lo, hi, S)
    how = dict(softcap=7.0, plan=plan)

    def step(x, stream=None):
        o, lse = fa.fa_fwd_scored(x["q"], x["k"], x["v"], False, 0.1, stream=stream, **how)
        g = fa.fa_bwd_scored(x["q"], x["k"], x["v"], o, x["dout"], lse, False, 0.1, stream=stream, **how)
        od, _ = fa.fa_decode_scored(x["q"][:, :, :1].contiguous(), x["k"], x["v"], _i32([S, 77]), 0.1, softcap=7.0,
                                    stream=stream)
        return (o, lse, *g[1:], od)

    want = [step(x) for x in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = []
        for x, s in zip(dev, streams):
            with torch.cuda.stream(s):
                got.append(step(x))
    torch.cuda.synchronize()
    _status_ok()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
