"""What is measured of the operators around the scores of an attention layer, each in its plain form (elementary torch
operations) and through the framework's entry points:

* ``prep``, ``prep_bwd``: norms of queries and keys for each head, position rotation with one or several axes, and the
  step from a projection's rows [token][head][channel] to head-major tensors or into a padded cache;
* ``mask``: documents, prefixes and windows as one interval of visible keys for each row;
* ``fwd``, ``train``: attention whose scores are capped by a tanh, biased by distance and masked by such intervals;
* ``decode``: the same for a single token of each request over a padded cache.

Formulas, for query row i at position p = i + Sk - Sq and key j:
  s = scale * <q, k>;  t = cap * tanh(s / cap);  z = t - slope_h * |p - j|;  O = softmax(z over lo <= j < hi) V."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF = torch.bfloat16


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one generated token for each of 48 running requests: its keys and values enter the cache
        dict(name="prep_step", op="prep", B=48, S=1, Hq=32, Hkv=8, d=128, rot=128, axes=1, inter=False, norm=True,
             offset=False, packed=True, room=1024, far=900),
        # the projections of a training batch of 2 x 8192 tokens
        dict(name="prep_batch", op="prep", B=2, S=8192, Hq=16, Hkv=16, d=128, rot=128, axes=1, inter=False, norm=True,
             offset=False, packed=True, room=0, far=0),
        # a small model's backward pass: half of the channels rotated, neighbours as pairs
        dict(name="prep_bwd_small", op="prep_bwd", B=2, S=300, Hq=4, Hkv=2, d=64, rot=32, axes=1, inter=True, norm=True,
             offset=True, packed=False, far=0),
        # images and video: three axes, grouped heads, an odd number of tokens
        dict(name="prep_bwd_axes", op="prep_bwd", B=3, S=2777, Hq=28, Hkv=4, d=128, rot=128, axes=3, inter=False,
             norm=True, offset=False, packed=True, far=200_000),
        # two short rows of a few documents with prefixes
        dict(name="mask_short", op="mask", B=2, S=777, docs=5, prefix=True, pad=True, causal=True, window=0),
        # one very long packed row
        dict(name="mask_long", op="mask", B=1, S=131_072, docs=300, prefix=True, pad=True, causal=True, window=4096),
        # the 2k training step with capped scores
        dict(name="train_capped", op="train", B=4, Hq=16, Hkv=16, Sq=2048, Sk=2048, d=128, docs=0, prefix=False,
             pad=False, causal=True, window=0, cap=50.0, slopes=False, mult=1.0),
        # 8k rows packed with documents, scores biased by distance, the rows' ends padded
        dict(name="train_docs", op="train", B=2, Hq=16, Hkv=16, Sq=8192, Sk=8192, d=128, docs=3, prefix=False,
             pad=True, causal=True, window=0, cap=0.0, slopes=True, mult=1.0),
        # prompts whose prefix is seen from everywhere, grouped heads, large scores under a cap
        dict(name="fwd_prefix", op="fwd", B=4, Hq=32, Hkv=8, Sq=4096, Sk=4096, d=128, docs=0, prefix=True, pad=False,
             causal=True, window=0, cap=30.0, slopes=False, mult=3.0),
        # a short chunk behind a cached prefix, with a window: latency counts
        dict(name="fwd_chunk", op="fwd", B=1, Hq=6, Hkv=3, Sq=130, Sk=513, d=64, docs=0, prefix=False, pad=False,
             causal=True, window=100, cap=0.0, slopes=True, mult=1.0),
        # one short request: latency counts
        dict(name="decode_one", op="decode", B=1, Hq=8, Hkv=2, lo=777, hi=777, d=64, window=0, cap=50.0, slopes=False,
             starts=False),
        # the ragged decode batch of the bf16 benchmark in a layer with a window of 4096 keys
        dict(name="decode_window", op="decode", B=32, Hq=32, Hkv=8, lo=1024, hi=32768, d=128, window=4096, cap=50.0,
             slopes=True, starts=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prep", "prep_bwd", "mask", "fwd", "fwd", "train", "train", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    if op in ("prep", "prep_bwd"):
        step = op == "prep" and rng.random() < 0.4
        most = 16384 * 48 * 128 // ((Hq + 2 * Hkv) * d)
        tokens = _spread(rng, 1, 256) if step else _spread(rng, 2, most)
        B = tokens if step else min(tokens, rng.choice([1, 2, 3, 8]))
        c = dict(op=op, B=B, S=tokens // B, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([0, 32, d // 2, d, d]),
                 axes=rng.choice([1, 1, 2, 3]), inter=rng.random() < 0.4, norm=rng.random() < 0.8,
                 offset=rng.random() < 0.3, packed=rng.random() < 0.6, far=rng.choice([0, 5000, 1_000_000]))
        if op == "prep":
            c["room"] = rng.choice([64, 300]) if step else 0
        return c
    cap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    slopes = rng.random() < 0.5
    window = rng.choice([0, 0, _spread(rng, 1, 6000)])
    if op == "mask":
        # the order of the documents is all that a seed gives this operator: enough of them that it differs
        S = _spread(rng, 64, 131_072)
        B = _spread(rng, 1, max(1, min(64, 131_072 // S)))
        return dict(op=op, B=B, S=S, docs=_spread(rng, 7, max(7, min(300, S // 8))), prefix=rng.random() < 0.5,
                    pad=rng.random() < 0.4, causal=rng.random() < 0.8, window=window and max(window, 16))
    if op == "decode":
        hi = _spread(rng, 1, 32768)
        most = max(1, min(64, 2 * 32768 * 32 * 8 * 128 // (3 * hi * Hkv * d)))
        return dict(op=op, B=_spread(rng, 1, most), Hq=Hq, Hkv=Hkv, lo=rng.randint(1, hi), hi=hi, d=d, window=window,
                    cap=cap, slopes=slopes, starts=rng.random() < 0.3)
    Sk = _spread(rng, 64 if op == "train" else 1, 8192)
    if op == "train" and window:  # with a single key in sight every gradient of a score is zero
        window = max(window, 32)
    most = max(1, min(16, 2 * 8192 * 8192 * 16 // (Sk * Sk * Hq)))
    docs = rng.choice([0, _spread(rng, 1, max(1, min(40, Sk)))])
    Sq = Sk if docs or op == "train" or rng.random() < 0.5 else rng.randint(1, Sk)
    return dict(op=op, B=_spread(rng, 1, most), Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, d=d, docs=docs,
                prefix=rng.random() < 0.4, pad=rng.random() < 0.3, causal=rng.random() < 0.8, window=window, cap=cap,
                slopes=slopes, mult=rng.choice([1.0, 1.0, 4.0]))


# ------------------------------------------------------------------ masks --

def _golden(n, phase):
    return [(phase + i * 0.6180339887498949) % 1.0 for i in range(n)]


def _documents(c, order):
    """Offsets of the documents over the flattened positions [B * Sk] and their prefixes (-1: padding), or
    (None, prefix of each batch row) or (None, None).  `order` permutes a row's documents (a padded one stays last)."""
    B, S = c["B"], c.get("Sk", c.get("S"))
    if not c["docs"]:
        if not c["prefix"]:
            return None, None
        return None, [int(f * (S + 1)) for f in _golden(B, 0.3)]
    cu, pre = [0], []
    for b in range(B):
        cuts = sorted(int(f * S) for f in _golden(c["docs"] - 1, 0.37 + 0.1 * b))
        lens = [y - x for x, y in zip([0] + cuts, cuts + [S])]
        docs = [(n, int(f * n) if c["prefix"] else 0) for n, f in zip(lens, _golden(len(lens), 0.2))]
        last = [(docs.pop()[0], -1)] if c["pad"] else []
        docs = [docs[i] for i in order(len(docs))] + last
        for n, p in docs:
            cu.append(cu[-1] + n)
            pre.append(p)
    return cu, (pre if c["prefix"] or c["pad"] else None)


def _intervals(c, cu, pre):
    """lo, hi [B, Sq] in numpy: the definition, row by row of the batch."""
    B, Sk = c["B"], c.get("Sk", c.get("S"))
    Sq = c.get("Sq", Sk)
    p = np.arange(Sq, dtype=np.int64) + Sk - Sq
    los, his = [], []
    for b in range(B):
        if cu is None:
            start, end = np.zeros(Sq, np.int64), np.full(Sq, Sk, np.int64)
            prefix = np.full(Sq, pre[b] if pre is not None else 0, np.int64)
        else:
            at = np.searchsorted(np.asarray(cu), b * Sk + p, side="right") - 1
            start = np.maximum(np.asarray(cu)[at] - b * Sk, 0)
            end = np.minimum(np.asarray(cu)[at + 1] - b * Sk, Sk)
            prefix = np.asarray(pre)[at] if pre is not None else np.zeros(Sq, np.int64)
        lo, hi = start, end
        if c["causal"]:
            hi = np.minimum(hi, np.maximum(p + 1, start + prefix))
        if c["window"]:
            lo = np.maximum(lo, p - c["window"] + 1)
            if not c["causal"]:
                hi = np.minimum(hi, p + c["window"])
        none = (prefix < 0) | (hi <= lo)
        los.append(np.where(none, 0, lo))
        his.append(np.where(none, 0, hi))
    return np.stack(los), np.stack(his)


def _plain_mask(s):
    B, Sk, Sq = s["B"], s["Sk"], s["Sq"]
    p = torch.arange(Sq, device=DEV) + (Sk - Sq)
    flat = torch.arange(B, device=DEV)[:, None] * Sk
    pre = s["prefix"]
    if s["cu"] is None:
        start = torch.zeros(B, Sq, dtype=torch.int64, device=DEV)
        end = torch.full((B, Sq), Sk, dtype=torch.int64, device=DEV)
        prefix = start if pre is None else pre.long()[:, None].expand(B, Sq)
    else:
        cu = s["cu"].long()
        at = torch.searchsorted(cu, flat + p, right=True) - 1
        start = (cu[at] - flat).clamp(min=0)
        end = (cu[at + 1] - flat).clamp(max=Sk)
        prefix = torch.zeros_like(start) if pre is None else pre.long()[at]
    lo, hi = start, end
    if s["causal"]:
        hi = torch.minimum(hi, torch.maximum(p + 1, start + prefix))
    if s["window"]:
        lo = torch.maximum(lo, p - s["window"] + 1)
        if not s["causal"]:
            hi = torch.minimum(hi, p + s["window"])
    none = (prefix < 0) | (hi <= lo)
    return dict(lo=torch.where(none, 0, lo).int(), hi=torch.where(none, 0, hi).int())


# ----------------------------------------------------------------- inputs --

def _lens(lo, hi, B, phase):
    """B lengths spread over [lo, hi], the same for every seed (their order is the seed's)."""
    return [lo + int(round(x * (hi - lo))) for x in _golden(B, phase)]


def _decode_lists(c):
    """Lengths of the requests and their first keys (a padded batch's rows start late)."""
    lens = _lens(c["lo"], c["hi"], c["B"], 0.25)
    return lens, [int(f * n * 0.5) if c["starts"] else 0 for f, n in zip(_golden(c["B"], 0.1), lens)]


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = np.random.RandomState(seed % (1 << 31))
    op, B = c["op"], c["B"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    randn = lambda *n: torch.randn(*n, generator=gen, device=DEV)  # noqa: E731
    s = dict(c)
    if op in ("mask", "fwd", "train"):
        s["Sk"] = c.get("Sk", c.get("S"))
        s["Sq"] = c.get("Sq", s["Sk"])
        cu, pre = _documents(c, lambda n: rnd.permutation(n).tolist())
        if cu is None and pre is not None:
            pre = [pre[i] for i in rnd.permutation(B)]
        s["cu"] = None if cu is None else i32(cu)
        s["prefix"] = None if pre is None else i32(pre)
        s["windowed"] = bool(c["window"] or pre is not None or cu is not None)
        if op == "mask":
            return s
        m = _plain_mask(s)
        s.update(lo=m["lo"], hi=m["hi"], plan=None)
        if own and s["windowed"]:  # a step's masks are planned once, for all of its layers
            import io_aware_exact_tcgen05_gb300 as fa
            lo, hi = fa.fa_row_bounds(B, s["Sq"], s["Sk"], c["causal"], window=c["window"], cu_docs=s["cu"],
                                      prefix=s["prefix"])
            s["plan"] = fa.fa_mask_plan(lo, hi, s["Sk"])
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    s["scale"] = 1.0 / math.sqrt(d)
    if op in ("fwd", "train"):
        s["q"] = (randn(B, Hq, s["Sq"], d) * c["mult"]).to(BF)
        s["k"], s["v"] = randn(B, Hkv, s["Sk"], d).to(BF), randn(B, Hkv, s["Sk"], d).to(BF)
        if op == "train":
            s["dout"] = randn(B, Hq, s["Sq"], d).to(BF)
        s["slope"] = _slopes(Hq) if c["slopes"] else None
        return s
    if op == "decode":
        lens, first = _decode_lists(c)
        order = rnd.permutation(B)
        lens, first = [lens[i] for i in order], [first[i] for i in order]
        s["seqlens"] = i32(lens)
        s["k_start"] = i32(first) if c["starts"] else None
        s["q"] = randn(B, Hq, 1, d).to(BF)
        for name in ("k", "v"):
            s[name] = torch.empty(B, Hkv, c["hi"], d, dtype=BF, device=DEV)
            for b in range(B):
                s[name][b] = randn(Hkv, c["hi"], d)
        s["slope"] = _slopes(Hq) if c["slopes"] else None
        return s
    # prep, prep_bwd: projections as a linear layer writes them, [token][head][channel]
    S, rot = c["S"], c["rot"]
    if c["packed"]:
        rows = (randn(B, S, Hq + 2 * Hkv, d) * torch.exp(0.5 * randn(1, 1, Hq + 2 * Hkv, 1))).to(BF)
        s["q"], s["k"], s["v"] = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = (randn(B, S, h, d).to(BF) for h in (Hq, Hkv, Hkv))
    s["inv_freq"] = None
    if rot:
        s["inv_freq"] = (1.0 / (500_000.0 ** (torch.arange(0, rot, 2, device=DEV).double() / rot))).float()
    s["freq_axis"] = None
    if rot and c["axes"] > 1:  # a share of the frequencies for each axis, one after another
        share = (torch.arange(rot // 2, device=DEV) * c["axes"]) // (rot // 2)
        s["freq_axis"] = share.to(torch.uint8)
    far = c["far"]
    if op == "prep" and c["room"]:
        at = [int(f * c["room"]) for f in _golden(B, 0.4)]
        s["row_start"] = i32([at[i] for i in rnd.permutation(B)])
        base = s["row_start"].long()[:, None] + torch.arange(S, device=DEV)
        s["k_cache"] = randn(B, Hkv, c["room"], d).to(BF)
        s["v_cache"] = randn(B, Hkv, c["room"], d).to(BF)
    else:
        s["row_start"] = None
        base = torch.arange(S, device=DEV).expand(B, S) + far
    wide = max(1, int(math.isqrt(S)))
    axes = [base] + [far // (a + 1) + (base // wide if a % 2 else base % wide) for a in range(1, c["axes"])]
    s["positions"] = torch.stack(axes).to(torch.int32).contiguous() if rot else None
    s["q_weight"] = s["k_weight"] = None
    if c["norm"]:
        mid = 0.0 if c["offset"] else 1.0
        s["q_weight"], s["k_weight"] = (mid + 0.2 * randn(d)).to(BF), (mid + 0.2 * randn(d)).to(BF)
    s["w_off"] = 1.0 if c["offset"] else 0.0
    if op == "prep_bwd":
        s["gq"], s["gk"], s["gv"] = (randn(B, h, S, d).to(BF) for h in (Hq, Hkv, Hkv))
    return s


# ------------------------------------------------------------ plain forms --

EPS = 1e-6


def _angles(s):
    """cos, sin [B, S, 1, rot / 2]; the products are formed in 64 bits: far positions lose their angle in 32."""
    pos = s["positions"].double()
    axis = torch.zeros(s["rot"] // 2, dtype=torch.int64, device=DEV) if s["freq_axis"] is None else s["freq_axis"].long()
    a = pos[axis].permute(1, 2, 0) * s["inv_freq"].double()
    return torch.cos(a)[:, :, None], torch.sin(a)[:, :, None]


def _rotate(x, s, cos, sin):
    """x [B, S, H, d], its first `rot` channels turned by the angles."""
    rot, half = s["rot"], s["rot"] // 2
    y = x.clone()
    if s["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _prep_one(x, w, s, trig):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + s["w_off"])
    if s["rot"]:
        x = _rotate(x, s, *trig)
    return x.transpose(1, 2).to(BF)


def _plain_prep(s):
    trig = [t.float() for t in _angles(s)] if s["rot"] else None
    q = _prep_one(s["q"], s["q_weight"], s, trig).contiguous()
    k, v = _prep_one(s["k"], s["k_weight"], s, trig), s["v"].transpose(1, 2)
    if s["row_start"] is None:
        return dict(q=q, k=k.contiguous(), v=v.contiguous())
    rows = s["row_start"].long()[:, None] + torch.arange(s["S"], device=DEV)
    b = torch.arange(s["B"], device=DEV)[:, None].expand_as(rows)
    fits = rows < s["room"]
    for cache, new in ((s["k_cache"], k), (s["v_cache"], v)):
        cache[b[fits], :, rows[fits]] = new.transpose(1, 2)[fits]
    return dict(q=q, k=s["k_cache"], v=s["v_cache"])


def _prep_back_one(x, w, g, s, trig):
    g = g.transpose(1, 2).float()
    if s["rot"]:
        g = _rotate(g, s, trig[0], -trig[1])
    if w is None:
        return g.to(BF), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).sum(dim=(0, 1, 2), dtype=torch.float64).float()
    a = g * (w.float() + s["w_off"])
    return (r * (a - n * (a * n).mean(-1, keepdim=True))).to(BF), dw


def _plain_prep_bwd(s):
    trig = [t.float() for t in _angles(s)] if s["rot"] else None
    dq, dwq = _prep_back_one(s["q"], s["q_weight"], s["gq"], s, trig)
    dk, dwk = _prep_back_one(s["k"], s["k_weight"], s["gk"], s, trig)
    out = dict(dq=dq, dk=dk, dv=s["gv"].transpose(1, 2).contiguous())
    if dwq is not None:
        out.update(dwq=dwq, dwk=dwk)
    return out


def _scores(q, k, lo, hi, s, h, first, positions):
    """z (hidden keys at -inf) and tanh(s / cap) of one head; keys first, first + 1, ..."""
    z = (q @ k.transpose(-1, -2)) * s["scale"]
    th = None
    if s["cap"]:
        th = torch.tanh(z / s["cap"])
        z = th * s["cap"]
    j = torch.arange(k.shape[0], device=DEV) + first
    if s["slope"] is not None:
        z = z - s["slope"][h].to(z.dtype) * (positions[:, None].to(z.dtype) - j.to(z.dtype)).abs()
    z = z.masked_fill((j < lo[:, None]) | (j >= hi[:, None]), -math.inf)
    return z, th


def _softmax(z):
    """Weights and log-sum-exp of each row; a row without keys gets zeros and -inf."""
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    return p, (m + torch.log(total))[:, 0]


def _attend(s, wide, back):
    """Forward (and backward) of every head in type `wide`; results in that type."""
    B, Hq, Sq, d = s["q"].shape
    Hkv, Sk = s["Hkv"], s["Sk"]
    group = Hq // Hkv
    pos = torch.arange(Sq, device=DEV) + (Sk - Sq)
    o = torch.empty(B, Hq, Sq, d, dtype=wide, device=DEV)
    lse = torch.empty(B, Hq, Sq, dtype=wide, device=DEV)
    out = dict(o=o, lse=lse)
    if back:
        out.update(dq=torch.empty_like(o), dk=torch.zeros(B, Hkv, Sk, d, dtype=wide, device=DEV),
                   dv=torch.zeros(B, Hkv, Sk, d, dtype=wide, device=DEV))
    for b in range(B):
        for h in range(Hq):
            q, k, v = (t.to(wide) for t in (s["q"][b, h], s["k"][b, h // group], s["v"][b, h // group]))
            z, th = _scores(q, k, s["lo"][b], s["hi"][b], s, h, 0, pos)
            p, lse[b, h] = _softmax(z)
            del z
            o[b, h] = p @ v
            if back:
                do = s["dout"][b, h].to(wide)
                out["dv"][b, h // group] += p.T @ do
                ds = p * (do @ v.T - (do * o[b, h]).sum(dim=1, keepdim=True))
                if th is not None:
                    ds = ds * (1 - th * th)
                out["dq"][b, h] = (ds @ k) * s["scale"]
                out["dk"][b, h // group] += (ds.T @ q) * s["scale"]
    return out


def _plain_attention(s):
    out = _attend(s, torch.float32, s["op"] == "train")
    return {n: t if n == "lse" else t.to(BF) for n, t in out.items()}


def _decode(s, wide):
    B, Hq, _, d = s["q"].shape
    group = Hq // s["Hkv"]
    o = torch.empty(B, Hq, 1, d, dtype=wide, device=DEV)
    lse = torch.empty(B, Hq, dtype=wide, device=DEV)
    lens = s["seqlens"].tolist()
    first = s["k_start"].tolist() if s["k_start"] is not None else [0] * B
    for b in range(B):
        n = lens[b]
        j0 = max(first[b], n - s["window"] if s["window"] else 0)
        j = torch.arange(j0, n, device=DEV)
        q = s["q"][b, :, 0].to(wide).view(s["Hkv"], group, d)
        k, v = s["k"][b, :, j0:n].to(wide), s["v"][b, :, j0:n].to(wide)
        z = (q @ k.transpose(1, 2)).reshape(Hq, n - j0) * s["scale"]
        if s["cap"]:
            z = s["cap"] * torch.tanh(z / s["cap"])
        if s["slope"] is not None:
            z = z - s["slope"].to(wide)[:, None] * (n - 1 - j).to(wide)
        p, lse[b] = _softmax(z)
        o[b, :, 0] = (p.view(s["Hkv"], group, n - j0) @ v).view(Hq, d)
    return dict(o=o, lse=lse)


def _plain_decode(s):
    out = _decode(s, torch.float32)
    return dict(o=out["o"].to(BF), lse=out["lse"])


# -------------------------------------------------------------- framework --

def _own(s):
    import io_aware_exact_tcgen05_gb300 as fa
    op = s["op"]
    if op == "mask":
        lo, hi = fa.fa_row_bounds(s["B"], s["Sq"], s["Sk"], s["causal"], window=s["window"], cu_docs=s["cu"],
                                  prefix=s["prefix"])
        return dict(lo=lo, hi=hi)
    if op == "decode":
        o, lse = fa.fa_decode_scored(s["q"], s["k"], s["v"], s["seqlens"], s["scale"], softcap=s["cap"],
                                     slopes=s["slope"], window=s["window"], k_start=s["k_start"])
        return dict(o=o, lse=lse)
    if op in ("fwd", "train"):
        how = dict(softcap=s["cap"], slopes=s["slope"], plan=s["plan"])
        causal = s["causal"] and s["plan"] is None  # a plan's intervals hold the causal rule already
        o, lse = fa.fa_fwd_scored(s["q"], s["k"], s["v"], causal, s["scale"], **how)
        if op == "fwd":
            return dict(o=o, lse=lse)
        dq, dk, dv = fa.fa_bwd_scored(s["q"], s["k"], s["v"], o, s["dout"], lse, causal, s["scale"], **how)
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    how = dict(positions=s["positions"], inv_freq=s["inv_freq"], freq_axis=s["freq_axis"], q_weight=s["q_weight"],
               k_weight=s["k_weight"], weight_offset=s["w_off"], eps=EPS, interleaved=s["inter"])
    if op == "prep":
        kept = dict(k_out=s["k_cache"], v_out=s["v_cache"], row_start=s["row_start"]) if s["room"] else {}
        q, k, v = fa.fa_qk_norm_rope(s["q"], s["k"], s["v"], **how, **kept)
        return dict(q=q, k=k, v=v)
    dq, dk, dv, dwq, dwk = fa.fa_qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["gv"], **how)
    out = dict(dq=dq, dk=dk, dv=dv)
    if dwq is not None:
        out.update(dwq=dwq, dwk=dwk)
    return out


def run(state):
    if own:
        return _own(state)
    return dict(prep=_plain_prep, prep_bwd=_plain_prep_bwd, mask=_plain_mask, fwd=_plain_attention,
                train=_plain_attention, decode=_plain_decode)[state["op"]](state)


def work(case):
    c = case
    op, B = c["op"], c["B"]
    if op == "mask":
        cu, pre = _documents(c, lambda n: list(range(n)))
        given = (len(cu) if cu is not None else 0) + (len(pre) if pre is not None else 0)
        return {"bytes": 8 * B * c["S"] + 4 * given, "flops": 0}
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if op in ("prep", "prep_bwd"):
        tokens, heads = B * c["S"], Hq + 2 * Hkv
        each = 2 * tokens * d
        small = 4 * c["axes"] * tokens + 2 * c["rot"] if c["rot"] else 0
        if op == "prep":
            return {"bytes": 2 * each * heads + small + (4 * d if c["norm"] else 0),
                    "flops": 8 * tokens * (Hq + Hkv) * d}
        x_read = each * (Hq + Hkv) + 4 * d + 8 * d if c["norm"] else 0
        return {"bytes": 2 * each * heads + x_read + small, "flops": 16 * tokens * (Hq + Hkv) * d}
    if op == "decode":
        keys = sum(min(n - x, c["window"] or n) for n, x in zip(*_decode_lists(c)))
        return {"bytes": 4 * keys * Hkv * d + 4 * B * Hq * d + 4 * B * Hq + 4 * B, "flops": 4 * keys * Hq * d}
    cu, pre = _documents(c, lambda n: list(range(n)))
    lo, hi = _intervals(c, cu, pre)
    pairs = int((hi - lo).sum()) * Hq
    rows, keys = B * Hq * c["Sq"], B * Hkv * c["Sk"]
    if op == "fwd":
        return {"bytes": 2 * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * d * pairs}
    return {"bytes": 2 * d * (4 * rows + 4 * keys) + 4 * rows, "flops": 14 * d * pairs}


# ---------------------------------------------------------------- 64 bits --

def _exact_prep(s, back):
    """Rotations as products of complex numbers, norms from the sums of squares, all in 64 bits."""
    rot, half = s["rot"], s["rot"] // 2
    turn = None
    if rot:
        pos = s["positions"].double()
        ang = torch.empty(s["B"], s["S"], half, dtype=torch.float64, device=DEV)
        for i in range(half):
            axis = 0 if s["freq_axis"] is None else int(s["freq_axis"][i])
            ang[..., i] = pos[axis] * float(s["inv_freq"][i])
        turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]

    def rotated(x, turn):
        if not rot:
            return x
        x = x.clone()
        if s["inter"]:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
            x[..., :rot] = torch.stack([z.real, z.imag], dim=-1).flatten(-2)
        else:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn
            x[..., :rot] = torch.cat([z.real, z.imag], dim=-1)
        return x

    res = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"]
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / s["d"] + EPS)
        if not back:
            u = x if w is None else (x / norm) * (w.double() + s["w_off"])
            res[n] = rotated(u, turn).permute(0, 2, 1, 3)
            continue
        g = rotated(s["g" + n].double().permute(0, 2, 1, 3), None if turn is None else turn.conj())
        if w is not None:
            unit = x / norm
            res["dw" + n] = (g * unit).flatten(0, 2).sum(0)
            g = g * (w.double() + s["w_off"])
            g = (g - unit * ((g * unit).sum(-1, keepdim=True) / s["d"])) / norm
        res["d" + n] = g
    if back:
        res["dv"] = s["gv"].double().permute(0, 2, 1, 3)
        return res
    res["v"] = s["v"].double().permute(0, 2, 1, 3)
    if s["row_start"] is not None:
        for n in ("k", "v"):
            cache = s[n + "_cache"].double()
            for b, at in enumerate(s["row_start"].tolist()):
                fit = max(0, min(s["S"], s["room"] - at))
                cache[b, :, at:at + fit] = res[n][b, :, :fit]
            res[n] = cache
    return res


def _exact_attention(s):
    """Each head from its definition, with the intervals rebuilt in numpy and the softmax's derivative taken through the
    normalised weights."""
    cu = None if s["cu"] is None else s["cu"].tolist()
    pre = None if s["prefix"] is None else s["prefix"].tolist()
    lo, hi = (torch.from_numpy(x).to(DEV) for x in _intervals(s, cu, pre))
    B, Hq, Sq, d = s["q"].shape
    Hkv, Sk, back = s["Hkv"], s["Sk"], s["op"] == "train"
    group, cap = Hq // Hkv, s["cap"]
    res = {n: torch.zeros(B, h, x, d, dtype=torch.float64, device=DEV)
           for n, h, x in (("o", Hq, Sq), ("dq", Hq, Sq), ("dk", Hkv, Sk), ("dv", Hkv, Sk)) if back or n == "o"}
    res["lse"] = torch.empty(B, Hq, Sq, dtype=torch.float64, device=DEV)
    j = torch.arange(Sk, device=DEV, dtype=torch.float64)
    for b in range(B):
        for h in range(Hq):
            kk, vv = s["k"][b, h // group].double(), s["v"][b, h // group].double()
            for r0 in range(0, Sq, 2048):
                rows = slice(r0, min(Sq, r0 + 2048))
                q = s["q"][b, h, rows].double()
                at = torch.arange(r0, r0 + q.shape[0], device=DEV, dtype=torch.float64) + (Sk - Sq)
                x = q.matmul(kk.t()).mul_(s["scale"])
                slack = None
                if cap:
                    x = torch.tanh(x / cap)
                    slack = 1 - x * x
                    x = x * cap
                if s["slope"] is not None:
                    x -= float(s["slope"][h]) * torch.abs(at[:, None] - j[None])
                seen = (j[None] >= lo[b, rows, None]) & (j[None] < hi[b, rows, None])
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                total = torch.logsumexp(x, dim=1)
                res["lse"][b, h, rows] = total
                w = torch.exp(x - torch.where(torch.isinf(total), torch.zeros_like(total), total)[:, None])
                del x, seen
                res["o"][b, h, rows] = w.matmul(vv)
                if back:
                    do = s["dout"][b, h, rows].double()
                    res["dv"][b, h // group] += w.t().matmul(do)
                    da = do.matmul(vv.t())
                    dx = w * (da - (w * da).sum(1, keepdim=True))
                    if cap:
                        dx = dx * slack
                    res["dq"][b, h, rows] = dx.matmul(kk) * s["scale"]
                    res["dk"][b, h // group] += dx.t().matmul(q) * s["scale"]
    return res


def _exact_decode(s):
    """One request and head at a time."""
    B, Hq, _, d = s["q"].shape
    group = Hq // s["Hkv"]
    res = dict(o=torch.zeros(B, Hq, 1, d, dtype=torch.float64, device=DEV),
               lse=torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV))
    for b, n in enumerate(s["seqlens"].tolist()):
        first = int(s["k_start"][b]) if s["k_start"] is not None else 0
        if s["window"]:
            first = max(first, n - s["window"])
        if first >= n:
            continue
        far = torch.arange(n - 1 - first, -1, -1, dtype=torch.float64, device=DEV)
        for hk in range(s["Hkv"]):
            k, v = s["k"][b, hk, first:n].double(), s["v"][b, hk, first:n].double()
            for h in range(hk * group, hk * group + group):
                x = k.matmul(s["q"][b, h, 0].double()) * s["scale"]
                if s["cap"]:
                    x = torch.tanh(x / s["cap"]) * s["cap"]
                if s["slope"] is not None:
                    x = x - float(s["slope"][h]) * far
                total = torch.logsumexp(x, dim=0)
                res["lse"][b, h] = total
                res["o"][b, h, 0] = torch.exp(x - total).matmul(v)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "mask":
        cu = None if s["cu"] is None else s["cu"].tolist()
        lo, hi = _intervals(s, cu, None if s["prefix"] is None else s["prefix"].tolist())
        return dict(lo=torch.from_numpy(lo).int().to(DEV), hi=torch.from_numpy(hi).int().to(DEV))
    if s["op"] == "decode":
        return _exact_decode(s)
    if s["op"] in ("fwd", "train"):
        return _exact_attention(s)
    return _exact_prep(s, s["op"] == "prep_bwd")
