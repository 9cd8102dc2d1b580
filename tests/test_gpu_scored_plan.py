"""Mask plans: what they hold, tile by tile, against the intervals they are made of; a plan of other sizes is refused, by
the binding where it knows the plan's and on the device otherwise."""

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads
from oracle import scored as so

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _plan(B, Sq, Sk, causal=True):
    return fa.fa_mask_plan(*fa.fa_row_bounds(B, Sq, Sk, causal), Sk)


@pytest.mark.parametrize("made,used", [
    # sizes whose plans have as many bytes: Sk within a tile, other rows and keys, another batch
    ((2, 300, 384), (2, 300, 300)), ((2, 300, 300), (2, 300, 384)), ((1, 46, 200), (1, 31, 500)),
    ((2, 20, 128), (1, 31, 500)), ((2, 5, 300), (1, 46, 200)),
])
@pytest.mark.parametrize("cap,d", [(0.0, 64), (5.0, 128)])
def test_a_plan_of_other_sizes_is_refused(made, used, cap, d):
    B, Sq, Sk = used
    assert fa.fa_mask_plan_size(*made) == fa.fa_mask_plan_size(*used)
    plan = _plan(*made)
    t = workloads.random_qkv(B, 4, 2, Sq, Sk, d, seed=1, with_dout=True)
    q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
    with pytest.raises(ValueError, match="plan was made for"):
        fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=cap, plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=cap, plan=_plan(*used))
    with pytest.raises(ValueError, match="plan was made for"):
        fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.1, softcap=cap, plan=plan)
    # a copy, of which the binding does not know the sizes; and no plan at all
    for other in (plan.clone(), torch.zeros_like(plan)):
        outs = [torch.full_like(x, 7.0) for x in (o, lse, q, k, v)]
        fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=cap, plan=other, o=outs[0], lse=outs[1])
        st, word = fa.fa_device_status(clear=True)
        assert st == fa.FA_ERR_INVALID_ARG and word & 0xffff == 4, hex(word)
        fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.1, softcap=cap, plan=other, dq=outs[2], dk=outs[3], dv=outs[4])
        st, word = fa.fa_device_status(clear=True)
        assert st == fa.FA_ERR_INVALID_ARG and word & 0xffff == 4, hex(word)
        for n in (0, 1, 3, 4):
            assert bool((outs[n] == 7.0).all()), n
    o1, l1 = fa.fa_fwd_scored(q, k, v, False, 0.1, softcap=cap, plan=_plan(*used).clone())
    assert torch.equal(o, o1) and torch.equal(lse, l1)
    assert fa.fa_device_status()[0] == 0


def test_split_calls_refuse_a_plan_of_other_sizes_too():
    # few rows with long keys; many heads on few keys: the joins read nothing out of range either
    for Hq, Hkv, Sq, Sk in ((2, 2, 100, 2500), (32, 1, 500, 130)):
        t = workloads.random_qkv(1, Hq, Hkv, Sq, Sk, 64, seed=2, with_dout=True)
        q, k, v, do = (t[n].to(DEV) for n in ("q", "k", "v", "dout"))
        o, lse = fa.fa_fwd_scored(q, k, v, True, 0.1)
        for other in (_plan(1, Sq, Sk - 1).clone(), torch.full((fa.fa_mask_plan_size(1, Sq, Sk),), 0x55, dtype=torch.uint8, device=DEV)):
            fa.fa_fwd_scored(q, k, v, False, 0.1, plan=other)
            assert fa.fa_device_status(clear=True)[0] == fa.FA_ERR_INVALID_ARG
            fa.fa_bwd_scored(q, k, v, o, do, lse, False, 0.1, plan=other)
            assert fa.fa_device_status(clear=True)[0] == fa.FA_ERR_INVALID_ARG
    assert fa.fa_device_status()[0] == 0


# ---------------------------------------------------------- what a plan holds --

def _bits(mask):
    """[n, 128] truth values -> [n, 4] words."""
    w = mask.reshape(len(mask), 4, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)
    return w.sum(-1).astype(np.uint32)


def _read(plan, B, Sq, Sk):
    nq, nk = -(-Sq // 128), -(-Sk // 128)
    np_ = -(-nq // 2)
    w = plan.cpu().numpy().view(np.int32)
    parts = [("sizes", (4,)), ("qt", (B, nq, 4)), ("gaps", (B, nq, 4)), ("seen", (B, nk, 4)), ("seen_causal", (B, nk, 4)), ("kt", (B, nk, 4)),
             ("rows", (B, Sq, 2)), ("by_q1", (B * nq,)), ("by_q2", (B * np_,)), ("by_k", (B * nk,)), ("by_k_row", (B, nk)),
             ("work", (B * (nq + np_ + nk),))]
    out, at = {}, 0
    for n, shape in parts:
        size = int(np.prod(shape))
        out[n] = w[at:at + size].reshape(shape)
        at += size
    assert at == len(w)
    return out


def _expected(lo, hi, Sk):
    """The same from the intervals, one tile after another."""
    B, Sq = lo.shape
    lo, hi = np.maximum(lo, 0), np.minimum(hi, Sk)
    none = hi <= lo
    lo, hi = np.where(none, 0, lo), np.where(none, 0, hi)
    nq, nk = -(-Sq // 128), -(-Sk // 128)
    pos, j = np.arange(Sq) + Sk - Sq, np.arange(nk * 128)
    r = dict(qt=np.zeros((B, nq, 4), int), gaps=np.zeros((B, nq, 4), int), kt=np.zeros((B, nk, 4), int), seen=np.zeros((B, nk, 4), np.uint32),
             seen_causal=np.zeros((B, nk, 4), np.uint32), rows=np.stack([lo, hi], -1))
    tiles = lambda a, b: -(-b // 128) - a // 128 if b > a else 0  # noqa: E731
    wq, wp, wk = np.zeros((B, nq), int), np.zeros((B, -(-nq // 2)), int), np.zeros((B, nk), int)
    for b in range(B):
        sees = (j >= lo[b][:, None]) & (j < hi[b][:, None])
        for n, s in (("seen", sees), ("seen_causal", sees & (j <= pos[:, None]))):
            all_rows = s.any(0).reshape(nk, 128)
            r[n][b] = _bits(all_rows)
            r["kt"][b, :, 2 if n == "seen" else 3] = np.where(all_rows.all(1), 0, 0x7fffffff)
        for t in range(nq):
            at = slice(t * 128, min(Sq, t * 128 + 128))
            live = hi[b, at] > lo[b, at]
            if live.any():
                l, h = lo[b, at][live].min(), hi[b, at].max()
                edges = np.flatnonzero(np.diff(sees[at].any(0)[l:h].astype(int))) + 1 + l  # of the keys that no row sees
                if len(edges) <= 4:
                    r["gaps"][b, t, :len(edges)] = edges
                r["qt"][b, t] = l, h, min(3, len(edges) // 2), (live & (hi[b, at] > pos[at] + 1)).any()
                if r["qt"][b, t, 3] and not (live & (lo[b, at] <= pos[at]) & (hi[b, at] > pos[at])).all():
                    r["qt"][b, t, 3] = 2
            wq[b, t] = tiles(*r["qt"][b, t, :2])
            wp[b, t // 2] += wq[b, t]
        for k in range(nk):
            meet = [t for t in range(nq) if r["qt"][b, t, 0] < k * 128 + 128 and r["qt"][b, t, 1] > k * 128]
            if meet:
                r["kt"][b, k, :2] = meet[0], meet[-1] + 1
            wk[b, k] = r["kt"][b, k, 1] - r["kt"][b, k, 0]
    # most work first; of equals the last query tile and the first key tile first
    late = lambda w: sorted(range(w.size), key=lambda e: (-w.flat[e], -e))  # noqa: E731
    early = lambda w: sorted(range(w.size), key=lambda e: (-w.flat[e], e))  # noqa: E731
    r.update(by_q1=late(wq), by_q2=late(wp), by_k=early(wk), work=np.concatenate([wq.ravel(), wp.ravel(), wk.ravel()]),
             by_k_row=[[b * nk + k for k in early(wk[b])] for b in range(B)])
    return r


def _intervals(kind, B, Sq, Sk):
    rng = np.random.RandomState(B + Sq + Sk)
    if kind == "documents":
        cu = [0] + sorted(rng.randint(0, B * Sk, 6).tolist()) + [B * Sk]
        return so.row_bounds(B, Sq, Sk, True, 0, cu, rng.randint(-1, 60, len(cu) - 1).tolist())
    if kind == "window":
        return so.row_bounds(B, Sq, Sk, False, 70)
    if kind == "none":
        return np.full((B, Sq), 5), np.full((B, Sq), 5)
    if kind == "scattered":  # never the last key of six, and rows without keys
        lo = rng.randint(-9, Sk // 6 + 1, (B, Sq)) * 6
        return lo, lo + rng.randint(-2, 5, (B, Sq))
    lo = rng.randint(-50, Sk, (B, Sq))  # any
    return lo, lo + rng.randint(-100, Sk, (B, Sq))


@pytest.mark.parametrize("kind", ["documents", "window", "none", "scattered", "any"])
@pytest.mark.parametrize("B,Sq,Sk", [(1, 1, 1), (2, 300, 300), (3, 129, 700), (1, 1500, 200), (2, 128, 256), (1, 4500, 4500)])
def test_a_plan_holds_what_its_intervals_say(kind, B, Sq, Sk):
    lo, hi = _intervals(kind, B, Sq, Sk)
    got = _read(fa.fa_mask_plan(*(torch.tensor(x.tolist(), dtype=torch.int32, device=DEV) for x in (lo, hi)), Sk), B, Sq, Sk)
    want = _expected(lo, hi, Sk)
    assert got["sizes"][:3].tolist() == [B, Sq, Sk]
    for n, x in want.items():
        x = np.asarray(x)
        assert np.array_equal(got[n].view(np.uint32) if x.dtype == np.uint32 else got[n], x), n
