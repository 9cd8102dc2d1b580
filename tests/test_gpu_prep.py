"""GPU parity of head norms with rotation (fa_qk_norm_rope and its backward) against the FP64 oracle, and of a layer
and a serving loop that run them with the attention.

Tolerances: outputs are rounded to bf16 once (half a step, 2^-8 of the value); before that fp32 arithmetic of a
dozen operations and sines off by 2^-20.5 leave 2^-19 of the sizes of what is added.  A weight's gradient is a sum
of n products in fp32: n 2^-24 of the sum of their magnitudes, and 2^-19 for the factors."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import scored as so
from tests.parity import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FINE = 2.0 ** -19


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _make(B, S, Hq, Hkv, d, rot, axes, norm, seed, far=0, packed=True, w_mid=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    t = {}
    if packed:
        rows = (rn(B, S, Hq + 2 * Hkv, d) * 2).to(BF).to(DEV)
        t["q"], t["k"], t["v"] = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
    else:  # head-major inputs, read in place
        t["q"], t["k"], t["v"] = ((rn(B, h, S, d) * 2).to(BF).to(DEV).transpose(1, 2) for h in (Hq, Hkv, Hkv))
    t["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2) / max(rot, 1))).float().to(DEV) if rot else None
    t["positions"] = None
    if rot:
        pos = torch.randint(-far, far + S + 1, (axes, B, S), generator=g, dtype=torch.int64)
        t["positions"] = _i32(pos)
    t["freq_axis"] = (torch.arange(rot // 2) % (axes + 1)).to(torch.uint8).to(DEV) if rot and axes > 1 else None
    t["qw"] = t["kw"] = None
    if norm:
        t["qw"], t["kw"] = ((w_mid + 0.3 * rn(d)).to(BF).to(DEV) for _ in range(2))
    return t


def _np(t):
    return None if t is None else to_np(t)


def _angles(t):
    if t["inv_freq"] is None:
        return None
    pos = t["positions"].cpu().numpy()
    pos = pos if pos.ndim == 3 else pos[None]
    return so.angles(pos, t["inv_freq"].cpu().numpy(), None if t["freq_axis"] is None else t["freq_axis"].cpu().numpy())


def _near(got, want, size, what, steps=2.0 ** -8):
    got = to_np(got)
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) - (steps * np.abs(want) * (1 + FINE) + FINE * size + 2.0 ** -120)
    assert over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, worst by {over.max():.3e}"


def _pair_size(x, w, w_off, eps, ang, rot, inter):
    """|a| + |b| of each output's pair."""
    u = so.norm_rope(x, w, w_off, eps, None, 0, inter)
    if not rot:
        return np.abs(u)
    size = np.abs(u)
    if inter:
        s = size[..., 0:rot:2] + size[..., 1:rot:2]
        size[..., 0:rot:2] = size[..., 1:rot:2] = s
    else:
        s = size[..., :rot // 2] + size[..., rot // 2:rot]
        size[..., :rot // 2] = size[..., rot // 2:rot] = s
    return size


CASES = [
    # B, S, Hq, Hkv, d, rot, axes, interleaved, norm, far, packed
    (1, 1, 1, 1, 64, 64, 1, False, True, 0, True),
    (2, 37, 4, 2, 128, 128, 1, False, True, 0, True),
    (1, 130, 5, 3, 64, 32, 1, True, True, 1000, False),
    (3, 50, 8, 1, 128, 48, 3, False, False, 2_000_000_000, True),
    (2, 19, 3, 3, 128, 16, 2, True, True, 1_000_000, True),
    (1, 257, 9, 2, 64, 0, 1, False, True, 0, False),
    (2, 11, 2, 2, 128, 0, 1, False, False, 0, True),
    (1, 2000, 6, 2, 128, 128, 2, True, False, 50_000, True),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("w_off", [0.0, 1.0])
def test_forward_and_backward(case, w_off):
    B, S, Hq, Hkv, d, rot, axes, inter, norm, far, packed = case
    t = _make(B, S, Hq, Hkv, d, rot, axes, norm, seed=21, far=far, packed=packed, w_mid=1.0 - w_off)
    how = dict(positions=t["positions"], inv_freq=t["inv_freq"], freq_axis=t["freq_axis"], q_weight=t["qw"],
               k_weight=t["kw"], weight_offset=w_off, eps=1e-5, interleaved=inter)
    if axes == 1 and rot:
        how["positions"] = t["positions"][0].contiguous()  # [B, S] is one axis
    q, k, v = fa.fa_qk_norm_rope(t["q"], t["k"], t["v"], **how)
    ang = _angles(t)
    for n, got in (("q", q), ("k", k)):
        x, w = to_np(t[n]), _np(t[n + "w"])
        _near(got, so.norm_rope(x, w, w_off, 1e-5, ang, rot, inter), _pair_size(x, w, w_off, 1e-5, ang, rot, inter), n)
    assert torch.equal(v, t["v"].transpose(1, 2))
    gen = torch.Generator().manual_seed(3)
    gq, gk, gv = (torch.randn(B, h, S, d, generator=gen).to(BF).to(DEV) for h in (Hq, Hkv, Hkv))
    rows = torch.full((B, S, Hq + 2 * Hkv, d), 9.0, dtype=BF, device=DEV)  # the packed projection's gradient
    outs = dict(dq=rows[:, :, :Hq], dk=rows[:, :, Hq:Hq + Hkv], dv=rows[:, :, Hq + Hkv:]) if packed else {}
    dq, dk, dv, dwq, dwk = fa.fa_qk_norm_rope_bwd(t["q"], t["k"], gq, gk, gv, **how, **outs)
    for n, got, dw, g in (("q", dq, dwq, gq), ("k", dk, dwk, gk)):
        x, w = to_np(t[n]), _np(t[n + "w"])
        dx, want, size, dw_size = so.norm_rope_bwd(x, w, w_off, 1e-5, ang, rot, inter, to_np(g))
        gs = np.abs(to_np(g)).transpose(0, 2, 1, 3)
        gs = gs + gs[..., ::-1] + np.roll(gs, rot // 2, -1) + np.roll(gs, -(rot // 2), -1) + np.roll(gs, 1, -1) + np.roll(gs, -1, -1)
        if w is not None:  # what turning g may be off by goes through a factor r (w + w_off) and the mean
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
            big = np.abs(w + w_off).max()
            gs = r * big * (gs + np.abs(x * r) * (gs * np.abs(x * r)).mean(-1, keepdims=True))
        _near(got, dx, size + gs, "d" + n)
        assert (dw is None) == (w is None)
        if w is not None:
            n_sum = x.shape[0] * x.shape[1] * x.shape[2]
            gx = (np.abs(to_np(g)).transpose(0, 2, 1, 3).max(-1, keepdims=True) * 2 * np.abs(x * r)).sum((0, 1, 2))
            tol = (n_sum * 2.0 ** -24 + FINE) * dw_size + FINE * gx
            assert np.all(np.abs(to_np(dw) - want) <= tol), "d" + n + "w"
    assert torch.equal(dv, gv.transpose(1, 2))
    if packed:
        assert dq.data_ptr() == rows.data_ptr() and not bool((rows == 9.0).all(-1).any())


def test_far_positions_keep_their_angles():
    # one pair, unit vector: the rotation itself, at the ends of the range of positions and frequencies
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123_456_789, 2 ** 24 + 1]
    freqs = [1.0, 2.0 ** -30, 0.1, 3.0e-5, 7.5, 1e5, 0.0, -0.3]
    S, d = len(pos), 64
    x = torch.zeros(1, S, 1, d, dtype=BF, device=DEV)
    x[..., :8] = 1.0
    f = torch.tensor(freqs, dtype=torch.float32, device=DEV)
    q, _, _ = fa.fa_qk_norm_rope(x, x, positions=_i32([pos]), inv_freq=f)
    ang = so.angles(np.array([[pos]]), np.array(freqs, np.float32), None)[0, :, 0]
    got = to_np(q)[0, 0]
    assert np.abs(got[:, :8] - np.cos(ang)).max() <= 2.0 ** -9 + 2.0 ** -19
    assert np.abs(got[:, 8:16] - np.sin(ang)).max() <= 2.0 ** -9 + 2.0 ** -19


def test_rows_of_a_cache():
    B, S, Hq, Hkv, d, room = 5, 3, 4, 2, 128, 40
    t = _make(B, S, Hq, Hkv, d, 64, 1, True, seed=23)
    start = [0, 37, 38, 39, -2]  # the last three lose rows past or before the cache
    kc, vc = (torch.full((B, Hkv, room, d), 5.0, dtype=BF, device=DEV) for _ in range(2))
    q, k, v = fa.fa_qk_norm_rope(t["q"], t["k"], t["v"], inv_freq=t["inv_freq"], q_weight=t["qw"], k_weight=t["kw"],
                                 k_out=kc, v_out=vc, row_start=_i32(start))
    assert k is kc and v is vc
    pos = np.array(start)[:, None] + np.arange(S)
    ang = so.angles(pos[None], t["inv_freq"].cpu().numpy(), None)
    want = so.norm_rope(to_np(t["k"]), _np(t["kw"]), 0.0, 1e-6, ang, 64, False)
    size = _pair_size(to_np(t["k"]), _np(t["kw"]), 0.0, 1e-6, ang, 64, False)
    left = torch.ones(B, room, dtype=torch.bool)
    for b in range(B):
        for s in range(S):
            if 0 <= pos[b, s] < room:
                _near(kc[b, :, pos[b, s]], want[b, :, s], size[b, :, s], "k")
                assert torch.equal(vc[b, :, pos[b, s]], t["v"][b, s])
                left[b, pos[b, s]] = False
    for c in (kc, vc):
        assert bool((c.transpose(1, 2)[left.to(DEV)] == 5.0).all())
    wq = so.norm_rope(to_np(t["q"]), _np(t["qw"]), 0.0, 1e-6, ang, 64, False)
    _near(q, wq, _pair_size(to_np(t["q"]), _np(t["qw"]), 0.0, 1e-6, ang, 64, False), "q")


def test_weights_gradients_are_the_same_every_time():
    t = _make(2, 700, 6, 2, 128, 128, 1, True, seed=24)
    g = [torch.randn(2, h, 700, 128, generator=torch.Generator().manual_seed(h)).to(BF).to(DEV) for h in (6, 2)]
    how = dict(positions=t["positions"], inv_freq=t["inv_freq"], q_weight=t["qw"], k_weight=t["kw"])
    a = fa.fa_qk_norm_rope_bwd(t["q"], t["k"], *g, **how)
    for _ in range(3):
        b = fa.fa_qk_norm_rope_bwd(t["q"], t["k"], *g, **how)
        assert all(torch.equal(x, y) for x, y in zip(a[:2] + a[3:], b[:2] + b[3:])) and b[2] is None


def test_only_one_weight_or_none():
    t = _make(1, 9, 2, 2, 64, 32, 1, True, seed=25)
    q, k, v = fa.fa_qk_norm_rope(t["q"], t["k"], positions=t["positions"], inv_freq=t["inv_freq"], q_weight=t["qw"])
    assert v is None
    _near(k, so.norm_rope(to_np(t["k"]), None, 0, 0, _angles(t), 32, False),
          _pair_size(to_np(t["k"]), None, 0, 0, None, 32, False), "k")
    g = torch.randn(1, 2, 9, 64).to(BF).to(DEV)
    out = fa.fa_qk_norm_rope_bwd(t["q"], None, g, g, positions=t["positions"], inv_freq=t["inv_freq"], q_weight=t["qw"])
    assert out[2] is None and out[3] is not None and out[4] is None
    # values that are not numbers stay with their token, head and pair
    x = t["k"].clone()
    x[0, 3, 1, 5] = float("nan")
    y = fa.fa_qk_norm_rope(t["q"], x, positions=t["positions"], inv_freq=t["inv_freq"])[1]
    bad = torch.isnan(y).nonzero().tolist()
    assert bad == [[0, 1, 3, 5], [0, 1, 3, 21]]


def test_head_major_and_strided_views_agree():
    t = _make(2, 65, 4, 2, 64, 64, 1, True, seed=26)
    how = dict(positions=t["positions"], inv_freq=t["inv_freq"], q_weight=t["qw"], k_weight=t["kw"])
    a = fa.fa_qk_norm_rope(t["q"], t["k"], t["v"], **how)
    hm = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (t["q"], t["k"], t["v"])]
    wide = torch.zeros(2, 70, 8, 96, dtype=BF, device=DEV)
    pad = [wide[:, 3:68, 4 * i:4 * i + h, 8:72].copy_(x) for i, (h, x) in enumerate(((4, t["q"]), (2, t["k"])))]
    for b in (fa.fa_qk_norm_rope(*hm, **how), fa.fa_qk_norm_rope(*pad, t["v"], **how)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    odd = torch.zeros(2, 65, 4, 65, dtype=BF, device=DEV)[..., :64]  # a stride that is no multiple of 8
    with pytest.raises(fa.FAError):
        fa.fa_qk_norm_rope(odd, t["k"], t["v"], **how)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(t["q"].transpose(2, 3), t["k"], t["v"], **how)


# ------------------------------------------------------- a layer, a serving loop --

def _layer_reference(x, B, S, Hq, Hkv, d, pos, inv_freq, qw, kw, lo, hi, cap, slopes, scale):
    """The layer in torch, 64 bits, differentiable."""
    def prep(y, w):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        a = (pos.double()[..., None] * inv_freq.double())[:, :, None]
        p, q = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([p * torch.cos(a) - q * torch.sin(a), q * torch.cos(a) + p * torch.sin(a)], -1).transpose(1, 2)
    q, k, v = prep(x[:, :, :Hq], qw), prep(x[:, :, Hq:Hq + Hkv], kw), x[:, :, Hq + Hkv:].transpose(1, 2)
    k, v = (y.repeat_interleave(Hq // Hkv, dim=1) for y in (k, v))
    t = cap * torch.tanh(q @ k.transpose(-1, -2) * scale / cap)
    j = torch.arange(S)
    z = t - slopes.double()[None, :, None, None] * (j[:, None] - j).abs()
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    w = torch.softmax(z.masked_fill(~seen[:, None], -1e30), -1) * seen[:, None]
    return w @ v


def test_training_layer_gradients():
    # projection rows -> norms and rotation -> capped, biased attention over documents -> and back
    B, S, Hq, Hkv, d = 2, 200, 4, 2, 64
    g = torch.Generator().manual_seed(31)
    rows = torch.randn(B, S, Hq + 2 * Hkv, d, generator=g).to(BF)
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).to(BF) for _ in range(2))
    dout = torch.randn(B, Hq, S, d, generator=g).to(BF)
    inv_freq = (1000.0 ** (-torch.arange(0, d, 2) / d)).float()
    cu, prefix = [0, 70, 180, 200, 330, 400], [0, 20, -1, 5, 0]
    lo, hi = so.row_bounds(B, S, S, True, 0, cu, prefix)
    starts = np.array([max(c for c in cu[:-1] if c <= x) for x in range(B * S)]).reshape(B, S)
    pos = torch.from_numpy(np.arange(B * S).reshape(B, S) - starts)  # positions restart with every document
    slopes = torch.tensor([0.2, 0.05, 0.01, 0.002])
    scale, cap = 1 / math.sqrt(d), 3.0

    dev = rows.to(DEV)
    q_in, k_in, v_in = dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv], dev[:, :, Hq + Hkv:]
    how = dict(positions=_i32(pos), inv_freq=inv_freq.to(DEV), q_weight=qw.to(DEV), k_weight=kw.to(DEV))
    q, k, v = fa.fa_qk_norm_rope(q_in, k_in, v_in, **how)
    plan = fa.fa_mask_plan(*fa.fa_row_bounds(B, S, S, True, cu_docs=_i32(cu), prefix=_i32(prefix)), S)
    att = dict(softcap=cap, slopes=slopes.to(DEV), plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, False, scale, **att)
    dq, dk, dv = fa.fa_bwd_scored(q, k, v, o, dout.to(DEV), lse, False, scale, **att)
    d_rows = torch.empty_like(dev)
    _, _, _, dqw, dkw = fa.fa_qk_norm_rope_bwd(q_in, k_in, dq, dk, dv, **how, dq=d_rows[:, :, :Hq],
                                               dk=d_rows[:, :, Hq:Hq + Hkv], dv=d_rows[:, :, Hq + Hkv:])
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0

    x = rows.double().requires_grad_()
    wq, wk = qw.double().requires_grad_(), kw.double().requires_grad_()
    ro = _layer_reference(x, B, S, Hq, Hkv, d, pos, inv_freq, wq, wk, torch.from_numpy(lo), torch.from_numpy(hi), cap,
                          slopes, scale)
    (ro * dout.double()).sum().backward()
    # Six roundings to bf16 on the way (q and k, weights, O, dS, dq, the result), each at most 2^-8 of its
    # value and independent: in the norm over a tensor less than sqrt(6) 2^-8 of it; twice that for the
    # differences dP - D, which are smaller than their terms.
    bound = 2 * math.sqrt(6) * 2.0 ** -8
    for n, got, ref in (("O", o, ro), ("rows", d_rows, x.grad), ("q weight", dqw, wq.grad), ("k weight", dkw, wk.grad)):
        ref = ref.detach()
        err = float((got.cpu().double() - ref).norm() / ref.norm())
        assert err <= bound, (n, err)
    # padding gets no gradient
    assert float(d_rows[0, 180:].abs().sum()) == 0.0


def test_serving_loop_matches_the_whole_prompt():
    # a prompt into the cache, then token by token; against one forward over all of them
    B, Hq, Hkv, d, room = 3, 8, 2, 128, 64
    lens, steps = [20, 1, 37], 5
    g = torch.Generator().manual_seed(33)
    rows = torch.randn(B, room, Hq + 2 * Hkv, d, generator=g).to(BF).to(DEV)
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).to(BF).to(DEV) for _ in range(2))
    inv_freq = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().to(DEV)
    how = dict(inv_freq=inv_freq, q_weight=qw, k_weight=kw)
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(Hq)], device=DEV)
    split = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])  # noqa: E731
    att = dict(softcap=20.0, slopes=slopes)
    q, k, v = fa.fa_qk_norm_rope(*split(rows), **how)
    whole, _ = fa.fa_fwd_scored(q, k, v, False, 0.09, **att,
                                plan=fa.fa_mask_plan(*fa.fa_row_bounds(B, room, room, True, window=24), room))
    kc, vc = (torch.zeros(B, Hkv, room, d, dtype=BF, device=DEV) for _ in range(2))
    for b in range(B):  # prompts of different lengths
        fa.fa_qk_norm_rope(*split(rows[b:b + 1, :lens[b]]), **how, k_out=kc[b:b + 1], v_out=vc[b:b + 1],
                           row_start=_i32([0]))
    n = _i32(lens)
    for s in range(steps):
        at = [x + s for x in lens]
        tok = torch.stack([rows[b, at[b]] for b in range(B)])[:, None]
        qs, _, _ = fa.fa_qk_norm_rope(*split(tok), **how, k_out=kc, v_out=vc, row_start=n)
        n = n + 1
        o, _ = fa.fa_decode_scored(qs, kc, vc, n, 0.09, **att, window=24)
        for b in range(B):
            assert torch.equal(kc[b, :, :at[b] + 1], k[b, :, :at[b] + 1])
            # the forward rounds weights to bf16 and their sum with them, the decode does not
            assert (o[b, :, 0].float() - whole[b, :, at[b]].float()).abs().max() <= 3 * 2.0 ** -8 * v.float().abs().max()
    assert fa.fa_device_status()[0] == 0
