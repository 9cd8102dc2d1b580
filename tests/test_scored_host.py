"""Host-side checks of the operators around the scores (no GPU): the oracle against independent statements of
its parts and against derivatives, and every refusal of the C ABI, which comes before any device call."""
import ctypes

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import build as fabuild
from oracle import scored as so

P, F, L = ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


# ---------------------------------------------------------------- oracle --

def _torch_attend(q, k, v, scale, seen, cap, slopes):
    B, Hq, Sq, d = q.shape
    Sk = k.shape[2]
    kk, vv = (x.repeat_interleave(Hq // k.shape[1], dim=1) for x in (k, v))
    t = q @ kk.transpose(-1, -2) * scale
    if cap:
        t = cap * torch.tanh(t / cap)
    dist = (torch.arange(Sq)[:, None] + Sk - Sq - torch.arange(Sk)).abs()
    z = t - torch.as_tensor(slopes)[None, :, None, None] * dist if slopes is not None else t
    z = z.masked_fill(~seen[:, None], -1e30)
    w = torch.softmax(z, -1) * seen[:, None]
    return w @ vv, torch.logsumexp(z, -1)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (1.5, False), (0.0, True), (2.0, True)])
def test_oracle_attention_and_gradients_match_autograd(cap, bias):
    rng = np.random.RandomState(3)
    B, Hq, Hkv, Sq, Sk, d = 2, 4, 2, 9, 13, 8
    q, k, v, do = (rng.randn(*s) for s in ((B, Hq, Sq, d), (B, Hkv, Sk, d), (B, Hkv, Sk, d), (B, Hq, Sq, d)))
    slopes = rng.rand(Hq) if bias else None
    lo, hi = so.row_bounds(B, Sq, Sk, True, window=5, cu=[0, 4, 13, 20, 26], prefix=[1, 3, -1, 2])
    assert (hi == lo).any() and (hi > lo).any()
    r = so.attend(q, k, v, 0.7, lo, hi, cap, slopes, do, bounds=True)
    seen = torch.from_numpy((np.arange(Sk) >= lo[..., None]) & (np.arange(Sk) < hi[..., None]))
    tq, tk, tv = (torch.from_numpy(x).requires_grad_() for x in (q, k, v))
    o, lse = _torch_attend(tq, tk, tv, 0.7, seen, cap, slopes)
    (o * torch.from_numpy(do)).sum().backward()
    live = seen.any(-1)[:, None].expand(B, Hq, Sq).numpy()
    np.testing.assert_allclose(r["o"], o.detach(), atol=1e-12)
    np.testing.assert_allclose(r["lse"][live], lse.detach().numpy()[live], atol=1e-12)
    assert np.all(r["lse"][~live] == -np.inf) and np.all(r["o"][~live] == 0)
    for n, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        np.testing.assert_allclose(r[n], t.grad, atol=1e-12)
        assert np.all(r["tol_" + n] > 0)


def test_oracle_gradients_match_differences():
    rng = np.random.RandomState(4)
    x = [rng.randn(1, 2, 4, 8), rng.randn(1, 1, 5, 8), rng.randn(1, 1, 5, 8)]
    do = rng.randn(1, 2, 4, 8)
    lo, hi = so.row_bounds(1, 4, 5, True, prefix=[2])
    slopes = np.array([0.3, 0.1])
    loss = lambda y: (so.attend(*y, 0.5, lo, hi, 1.2, slopes)["o"] * do).sum()  # noqa: E731
    r = so.attend(*x, 0.5, lo, hi, 1.2, slopes, do)
    for i, n in enumerate(("dq", "dk", "dv")):
        for at in [tuple(rng.randint(s) for s in x[i].shape) for _ in range(6)]:
            hi_x, lo_x = [y.copy() for y in x], [y.copy() for y in x]
            hi_x[i][at] += 1e-5
            lo_x[i][at] -= 1e-5
            assert abs((loss(hi_x) - loss(lo_x)) / 2e-5 - r[n][at]) < 1e-8


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [0, 1, 4])
def test_oracle_row_bounds_are_the_masks_they_stand_for(causal, window):
    # visibility stated key by key: same document, causal or in the document's prefix, within the window
    B, S, cu, pre = 2, 12, [0, 5, 5, 9, 16, 21], [2, 0, -1, 3, 0]
    lo, hi = so.row_bounds(B, S, S, causal, window, cu, pre)
    doc = [max([d for d in range(5) if cu[d] <= x < cu[d + 1]], default=None) if x < 21 else None for x in range(B * S)]
    for b in range(B):
        for i in range(S):
            want = []
            di = doc[b * S + i]
            for j in range(S):
                if di is None or doc[b * S + j] != di or pre[di] < 0:
                    continue
                in_prefix = b * S + j < max(cu[di], b * S) + pre[di]
                if causal and not (j <= i or in_prefix):
                    continue
                if window and (j < i - window + 1 or (not causal and j >= i + window)):
                    continue
                want.append(j)
            assert list(range(lo[b, i], hi[b, i])) == want, (b, i)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_oracle_norm_rope_matches_autograd(inter, rot):
    rng = np.random.RandomState(5)
    B, S, H, d = 2, 3, 2, 8
    x, w, dy = rng.randn(B, S, H, d), rng.randn(d), rng.randn(B, H, S, d)
    pos = rng.randint(-5, 100, (2, B, S))
    f = (0.9 ** np.arange(rot // 2)).astype(np.float32)
    ax = np.arange(rot // 2) % 3  # axis 2 is not there: those do not turn
    ang = so.angles(pos, f, ax)
    tx, tw = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    u = tx * torch.rsqrt((tx * tx).mean(-1, keepdim=True) + 1e-3) * (tw + 0.5)
    a = torch.zeros(B, S, 1, rot // 2, dtype=torch.float64)
    for i in range(rot // 2):
        if ax[i] < 2:
            a[:, :, 0, i] = torch.from_numpy(pos[ax[i]]).double() * float(f[i])
    pieces = list(u.unbind(-1))
    for i in range(rot // 2):
        m, n = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = torch.cos(a[..., i]), torch.sin(a[..., i])
        pieces[m], pieces[n] = u[..., m] * c - u[..., n] * s, u[..., n] * c + u[..., m] * s
    y = torch.stack(pieces, -1).transpose(1, 2)
    (y * torch.from_numpy(dy)).sum().backward()
    np.testing.assert_allclose(so.norm_rope(x, w, 0.5, 1e-3, ang, rot, inter), y.detach(), atol=1e-12)
    dx, dw, size, dw_size = so.norm_rope_bwd(x, w, 0.5, 1e-3, ang, rot, inter, dy)
    np.testing.assert_allclose(dx, tx.grad, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad, atol=1e-11)
    assert np.all(size >= np.abs(dx) - 1e-12) and np.all(dw_size >= np.abs(dw) - 1e-12)


def test_oracle_angles_are_exact_far_out():
    # 2^31 - 1 positions at 1 radian each, against the angle in 80-digit arithmetic
    a = so.angles(np.array([[[2 ** 31 - 1]]]), np.array([1.0], np.float32), None)[0, 0, 0, 0]
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = 2 * Decimal(so._PI_DIGITS[0] + "." + so._PI_DIGITS[1:])
    want = Decimal(2 ** 31 - 1) % two_pi
    assert abs(Decimal(a) - want) < Decimal(1e-14) * 10


# ---------------------------------------------------------------- refusals --

def _fwd(lib, q=16, lse=None, B=1, Hq=2, Hkv=2, Sq=8, Sk=8, d=128, scale=0.1, cap=0.0, slopes=None, plan=None,
         nplan=0, ws=None, nws=0):
    return lib.fa_fwd_scored(P(q), P(16), P(16), P(16), P(lse), B, Hq, Hkv, Sq, Sk, d, 1, F(scale), F(cap),
                             P(slopes), P(plan), nplan, P(ws), nws, None)


def test_scored_attention_refuses_before_any_device_call(lib):
    assert _fwd(lib, B=0) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, Hq=3, Hkv=2) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, d=96) == fa.FA_ERR_UNSUPPORTED
    assert _fwd(lib, q=8) == fa.FA_ERR_INVALID_ARG
    for scale in (float("nan"), float("inf"), -0.5):
        assert _fwd(lib, scale=scale) == fa.FA_ERR_INVALID_ARG
    for cap in (-1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21):
        assert _fwd(lib, cap=cap) == fa.FA_ERR_INVALID_ARG
        assert b"softcap" in lib.fa_last_error_detail()
    assert _fwd(lib, scale=3e38, cap=2.0 ** -20) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, slopes=18) == fa.FA_ERR_INVALID_ARG
    need = fa.fa_mask_plan_size(1, 8, 8)
    assert _fwd(lib, plan=256, nplan=need - 1) == fa.FA_ERR_WORKSPACE
    split = fa.fa_fwd_scored_workspace_size(1, 2, 2, 8, 5000, 128)  # few rows, long keys
    assert split > 0 == fa.fa_fwd_scored_workspace_size(1, 2, 2, 8, 600, 128) == fa.fa_fwd_scored_workspace_size(
        8, 32, 8, 4096, 4096, 128) == fa.fa_fwd_scored_workspace_size(1, 3, 2, 8, 5000, 128)
    assert _fwd(lib, Sk=5000, ws=256, nws=split - 1) == fa.FA_ERR_WORKSPACE
    plain = fa.fa_bwd_workspace_size(1, 32, 512, 128)  # enough for any call; many heads on few keys may use more
    assert fa.fa_bwd_scored_workspace_size(1, 32, 2, 512, 512, 128) > plain == fa.fa_bwd_scored_workspace_size(
        1, 32, 32, 512, 512, 128)
    assert _fwd(lib, Sk=5000, ws=264, nws=split) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, plan=260, nplan=need) == fa.FA_ERR_INVALID_ARG

    def bwd(ws=256, nws=1 << 20, cap=0.0, plan=None, nplan=0):
        return lib.fa_bwd_scored(*[P(16)] * 9, 1, 2, 2, 8, 8, 128, 1, F(0.1), F(cap), None, P(plan), nplan, P(ws), nws,
                                 None)
    assert bwd(nws=16) == fa.FA_ERR_WORKSPACE
    assert bwd(ws=0) == fa.FA_ERR_WORKSPACE
    assert bwd(cap=-1.0) == fa.FA_ERR_INVALID_ARG
    assert bwd(plan=256, nplan=1) == fa.FA_ERR_WORKSPACE

    def dec(seqlens=16, B=2, Hkv=2, Sk=100, window=0, ws=256, nws=1 << 24, k_start=None, cap=0.0):
        return lib.fa_decode_scored(P(16), P(16), P(16), P(16), None, P(seqlens), P(k_start), B, 4, Hkv, Sk, 128,
                                    F(0.1), F(cap), None, window, P(ws), nws, None)
    assert dec(seqlens=0) == fa.FA_ERR_INVALID_ARG
    assert dec(Hkv=3) == fa.FA_ERR_INVALID_ARG
    assert dec(window=-1) == fa.FA_ERR_INVALID_ARG
    assert dec(k_start=18) == fa.FA_ERR_INVALID_ARG
    assert dec(Sk=1000, nws=64) == dec(Sk=1000, ws=0) == fa.FA_ERR_WORKSPACE
    assert fa.fa_decode_scored_workspace_size(2, 4, 2, 100, 128) == 0 < fa.fa_decode_scored_workspace_size(2, 4, 2, 1000, 128)
    assert fa.fa_decode_scored_workspace_size(2, 4, 2, 1000, 128, 256) == 0  # a short window
    assert dec(cap=float("nan")) == fa.FA_ERR_INVALID_ARG
    assert dec(B=1 << 29, Sk=1, nws=1 << 60) == fa.FA_ERR_INVALID_ARG  # B x Hq past 32 bits
    assert fa.fa_decode_scored_workspace_size(0, 1, 1, 8, 64) == 0
    assert fa.fa_decode_scored_workspace_size(2, 4, 2, 100000, 128, 64) < fa.fa_decode_scored_workspace_size(
        2, 4, 2, 100000, 128)


def test_masks_refuse_before_any_device_call(lib):
    def rows(lo=16, hi=16, cu=None, pre=None, n=0, B=1, Sq=8, Sk=8, window=0):
        return lib.fa_row_bounds(P(cu), P(pre), n, P(lo), P(hi), B, Sq, Sk, 1, window, None)
    assert rows(B=0) == rows(Sq=0) == rows(Sk=-1) == fa.FA_ERR_INVALID_ARG
    assert rows(B=65536) == fa.FA_ERR_INVALID_ARG
    assert rows(B=2, Sk=1 << 30) == fa.FA_ERR_INVALID_ARG
    assert rows(lo=0) == rows(hi=18) == fa.FA_ERR_INVALID_ARG
    assert rows(cu=16, n=0) == fa.FA_ERR_INVALID_ARG
    assert rows(cu=17, n=1) == rows(pre=17) == fa.FA_ERR_INVALID_ARG
    assert rows(window=-1) == fa.FA_ERR_INVALID_ARG
    need = fa.fa_mask_plan_size(2, 300, 400)
    assert fa.fa_mask_plan_size(0, 1, 1) == 0 and need >= 2 * 300 * 8
    plan = lambda ptr, n: lib.fa_mask_plan(P(16), P(16), 2, 300, 400, P(ptr), n, None)  # noqa: E731
    assert plan(256, need - 1) == plan(0, need) == fa.FA_ERR_WORKSPACE
    assert plan(264, need) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_mask_plan(None, P(16), 2, 300, 400, P(256), need, None) == fa.FA_ERR_INVALID_ARG


def _view(ptr=16, sb=1024, st=512, sh=128):
    return fa._Heads(ptr, sb, st, sh)


def _prep(lib, q=None, k=None, v=None, q_out=16, k_out=16, v_out=None, row_start=None, S_out=2, qw=None, eps=1e-6,
          w_off=0.0, pos=None, axes=1, freq=16, rot=128, B=2, S=2, Hq=4, Hkv=4, d=128):
    return lib.fa_qk_norm_rope(q or _view(), k or _view(), v, P(q_out), P(k_out), P(v_out), P(row_start), S_out, P(qw),
                               None, F(w_off), F(eps), P(pos), axes, P(freq), None, rot, 0, B, S, Hq, Hkv, d, None)


def test_norm_rope_refuses_before_any_device_call(lib):
    bad = fa.FA_ERR_INVALID_ARG
    assert _prep(lib, B=0) == _prep(lib, Hq=0) == bad
    assert _prep(lib, d=80) == fa.FA_ERR_UNSUPPORTED
    assert _prep(lib, rot=24) == _prep(lib, rot=144) == _prep(lib, rot=-16) == bad
    assert _prep(lib, rot=64, d=64, freq=0) == bad
    assert _prep(lib, axes=0) == _prep(lib, axes=256) == _prep(lib, pos=18) == bad
    assert _prep(lib, eps=-1.0) == _prep(lib, eps=float("nan")) == _prep(lib, w_off=float("inf")) == bad
    assert _prep(lib, q=_view(ptr=8)) == _prep(lib, q=_view(ptr=0)) == bad
    assert _prep(lib, k=_view(sb=1020)) == _prep(lib, k=_view(sh=-128)) == _prep(lib, k=_view(st=1 << 41)) == bad
    assert _prep(lib, q_out=0) == _prep(lib, k_out=20) == _prep(lib, qw=8) == bad
    assert _prep(lib, v=_view()) == _prep(lib, v_out=16) == bad
    assert _prep(lib, S_out=1) == _prep(lib, S_out=0, row_start=16) == _prep(lib, row_start=18) == bad
    assert _prep(lib, B=1 << 20, S=1 << 11, S_out=1 << 11) == bad

    def back(dq=None, dk=None, dv=None, dv_out=None, dqw=None, qw=None, ws=256, nws=1 << 20):
        return lib.fa_qk_norm_rope_bwd(_view(), _view(), P(16), P(16), P(dv_out), dq or _view(), dk or _view(), dv,
                                       P(dqw), None, P(qw), None, F(0.0), F(1e-6), None, 1, P(16), None, 128, 0, 2, 2, 4,
                                       4, 128, P(ws), nws, None)
    for v in (_view(st=384), _view(sb=512), _view(sh=0), _view(sb=0)):  # written views that overlap themselves
        assert back(dq=v) == bad
        assert b"overlaps itself" in lib.fa_last_error_detail()
    assert back(dv=_view()) == back(dv_out=16) == bad
    assert back(dqw=16) == bad  # a gradient of a weight that is not there
    assert back(dqw=16, qw=16, nws=64) == back(dqw=16, qw=16, ws=0) == fa.FA_ERR_WORKSPACE
    assert fa.fa_qk_norm_rope_bwd_workspace_size(128) >= 128 * 4


def test_binding_refuses_what_is_no_cuda_tensor():
    x = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fa.fa_fwd_scored(x, x, x, True, 0.1)
    with pytest.raises(TypeError):
        fa.fa_decode_scored(x[:, :, :1], x, x, torch.zeros(1, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        fa.fa_decode_scored(x, x, x, torch.zeros(1, dtype=torch.int32), 0.1)
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(x, x)
    with pytest.raises(TypeError):
        fa.fa_mask_plan(torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        fa.fa_row_bounds(0, 8, 8, True)
    with pytest.raises(ValueError):
        fa.fa_row_bounds(1, 1 << 33, 8, True)
