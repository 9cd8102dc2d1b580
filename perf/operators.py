"""What is measured of the paged 8-bit KV cache: each operator in its plain form (elementary torch operations) and
through the framework's entry points, on cases from one request to long ragged batches.

The cache holds e4m3 codes [pages, Hkv, page, d] with one scale for each (page, KV head): a value is code * scale.
Requests own pages through a block table [B, max_blocks].  ``k_bounds`` holds, for each (page, KV head) and channel,
the largest and the smallest key code in units of 4, rounded outwards (int8)."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one generated token for each of 64 running requests: the slot map of a decode step
        dict(name="assign_step", op="assign", B=64, lo=1, hi=8191, new_lo=1, new_hi=1, page=16),
        # a batch of new prompts behind cached prefixes
        dict(name="assign_prompts", op="assign", B=48, lo=0, hi=6000, new_lo=1, new_hi=4096, page=64),
        # the keys and values of one generated token for each of 96 requests
        dict(name="write_step", op="write", B=96, lo=1, hi=2000, new_lo=1, new_hi=1, Hkv=8, d=128, page=64,
             bounds=True, token_major=True),
        # prompts of up to 8k tokens entering the cache, K and V as slices of one projection's output
        dict(name="write_prompts", op="write", B=16, lo=0, hi=300, new_lo=1, new_hi=8192, Hkv=8, d=128, page=64,
             bounds=True, token_major=True),
        # one short request: latency counts
        dict(name="decode_one", op="decode", B=1, lo=777, hi=777, Sq=1, Hq=8, Hkv=2, d=64, page=16, chosen=0),
        # the ragged decode batch of the bf16 benchmark, from the 8-bit cache
        dict(name="decode_ragged", op="decode", B=32, lo=1024, hi=32768, Sq=1, Hq=32, Hkv=8, d=128, page=64,
             chosen=0),
        # four drafted tokens for each request checked in one pass
        dict(name="decode_verify", op="decode", B=24, lo=500, hi=9000, Sq=4, Hq=32, Hkv=4, d=128, page=32,
             chosen=0),
        # long contexts of which 64 blocks of 64 tokens are attended
        dict(name="decode_chosen", op="decode", B=8, lo=40001, hi=65536, Sq=1, Hq=32, Hkv=8, d=128, page=64,
             chosen=64),
        # choosing the blocks of short contexts and small pages
        dict(name="select_short", op="select", B=5, lo=100, hi=3001, Sq=1, Hq=16, Hkv=2, d=64, page=16, chosen=24),
        # choosing 64 of up to 2048 blocks for each KV head of a long batch
        dict(name="select_long", op="select", B=8, lo=70000, hi=131072, Sq=1, Hq=32, Hkv=8, d=128, page=64,
             chosen=64),
        # a few short cached prefixes handed to the prompt's attention
        dict(name="read_short", op="read", B=3, lo=1, hi=700, Hkv=2, d=64, page=16),
        # long cached prefixes handed to the prompt's attention
        dict(name="read_long", op="read", B=4, lo=9001, hi=40000, Hkv=8, d=128, page=64),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "write", "decode", "decode", "select", "read"])
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "assign":
        hi = _spread(rng, 1, 9000)
        new = rng.choice([1, _spread(rng, 2, 4096)])
        return dict(op=op, B=_spread(rng, 1, 256 if new == 1 else 32), lo=rng.randint(0, hi), hi=hi, new_lo=1,
                    new_hi=new, page=page)
    if op == "write":
        hi = _spread(rng, 1, 2000)
        new = rng.choice([1, _spread(rng, 2, 8000)])
        return dict(op=op, B=_spread(rng, 1, 256 if new == 1 else 15), lo=rng.randint(0, hi), hi=hi, new_lo=1,
                    new_hi=new, Hkv=Hkv, d=d, page=page, bounds=rng.random() < 0.5,
                    token_major=rng.random() < 0.5)
    if op == "decode":
        hi = _spread(rng, 1, 60000)
        chosen = rng.choice([0, 0, _spread(rng, 4, 96)])
        most = max(1, min(64, 500_000 // hi))
        return dict(op=op, B=_spread(rng, 1, most), lo=rng.randint(1, hi), hi=hi, Sq=rng.choice([1, 1, 2, 3, 5]),
                    Hq=Hkv * group, Hkv=Hkv, d=d, page=page, chosen=chosen)
    if op == "select":
        hi = _spread(rng, 50, 130_000)
        most = max(1, min(64, 1_000_000 // hi))
        return dict(op=op, B=_spread(rng, 1, most), lo=rng.randint(1, hi), hi=hi, Sq=rng.choice([1, 1, 2, 4]),
                    Hq=Hkv * group, Hkv=Hkv, d=d, page=page, chosen=_spread(rng, 4, 128))
    hi = _spread(rng, 1, 40000)
    most = max(1, min(64, 100_000 // hi))
    return dict(op=op, B=_spread(rng, 1, most), lo=rng.randint(1, hi), hi=hi, Hkv=Hkv, d=d, page=page)


def _lens(lo, hi, B, phase):
    """B lengths spread over [lo, hi], the same for every seed (their order is the seed's)."""
    f = [(phase + i * 0.6180339887498949) % 1.0 for i in range(B)]
    return [lo + int(round(x * (hi - lo))) for x in f]


def _len_lists(c):
    old = _lens(c["lo"], c["hi"], c["B"], 0.25)
    new = _lens(c["new_lo"], c["new_hi"], c["B"], 0.5) if "new_lo" in c else [0] * c["B"]
    return old, new


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], exactly (a power function may be off in its last bit)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pages(n, ps):
    return (n + ps - 1) // ps


# ----------------------------------------------------------------- inputs --

def _quantise(x):
    """codes, scale of x [pages, heads, page, d]: the smallest power of two with which the largest value fits."""
    m, ex = torch.frexp(x.abs().amax(dim=(2, 3)))
    e = (ex - 9 + (m > 0.875).int()).clamp(-100, 119)
    scale = _pow2(e)
    return (x / scale[:, :, None, None]).clamp_(-448, 448).to(F8), scale


def _cache(gen, pages, heads, ps, d, spread):
    """One cache tensor as a model fills it: channels of unequal size, tokens of unequal norm."""
    channel = torch.exp(spread * torch.randn(heads, 1, d, generator=gen, device=DEV))
    x = torch.randn(pages, heads, ps, d, generator=gen, device=DEV)
    x *= channel
    x *= torch.exp(0.2 * torch.randn(pages, heads, ps, 1, generator=gen, device=DEV))
    return _quantise(x)


def _bounds_of(codes):
    v = codes.float() / 4
    return torch.stack([torch.ceil(v.amax(dim=2)), torch.floor(v.amin(dim=2))], dim=2).to(torch.int8)


def _tables(gen, order, lens, room, ps, extra):
    """Block tables [B, max_blocks] over a shuffled pool of pages, -1 behind each request's last page."""
    n = [_pages(x, ps) for x in lens]
    total = sum(n) + extra
    pool = torch.randperm(max(total, 1), generator=gen, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), max(room, 1)), -1, dtype=torch.int32)
    at = 0
    for b in order:
        table[b, :n[b]] = pool[at:at + n[b]]
        at += n[b]
    return table.to(DEV), pool[at:].to(DEV), max(total, 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ps, B, op = c["page"], c["B"], c["op"]
    old, new = _len_lists(c)
    order = np.random.RandomState(seed % (1 << 31)).permutation(B).tolist()
    old, new = [old[i] for i in order], [new[i] for i in order]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(op=op, ps=ps, B=B, seqlens=i32(old))
    room = max(_pages(a + b, ps) for a, b in zip(old, new))
    grow = sum(_pages(a + b, ps) - _pages(a, ps) for a, b in zip(old, new))
    table, free, pages = _tables(gen, order, old, room, ps, grow + (7 if op == "assign" else 0))
    s.update(table=table, pages=pages)
    if op == "assign":
        s.update(newlens=i32(new), free=free, total=sum(new))
        return s
    Hkv, d = c["Hkv"], c["d"]
    if op == "write":
        # the slots of the new tokens, as the assign call hands them out
        tab, at, slots = table.cpu(), 0, []
        free_cpu = free.cpu()
        for b in range(B):
            n0, n1 = _pages(old[b], ps), _pages(old[b] + new[b], ps)
            tab[b, n0:n1] = free_cpu[at:at + n1 - n0]
            at += n1 - n0
            pos = torch.arange(old[b], old[b] + new[b])
            slots.append(tab[b][pos // ps].long() * ps + pos % ps)
        s["slots"] = torch.cat(slots).to(DEV)
        s["k_cache"], s["k_scale"] = _cache(gen, pages, Hkv, ps, d, 0.5)
        s["v_cache"], s["v_scale"] = _cache(gen, pages, Hkv, ps, d, 0.2)
        s["k_bounds"] = _bounds_of(s["k_cache"]) if c["bounds"] else None
        n = sum(new)
        kv = torch.randn(2, n, Hkv, d, generator=gen, device=DEV)
        kv *= torch.exp(0.6 * torch.randn(2, 1, Hkv, d, generator=gen, device=DEV))
        kv = kv.to(torch.bfloat16)
        if c["token_major"]:  # rows [token][K heads, V heads]: both are strided views of it
            kv = kv.transpose(0, 1).contiguous()
            s["k"], s["v"] = kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)
        else:
            s["k"], s["v"] = kv[0].transpose(0, 1).contiguous(), kv[1].transpose(0, 1).contiguous()
        return s
    if op == "select":
        # summaries of pages whose keys drift along the sequence
        channel = torch.exp(0.5 * torch.randn(Hkv, d, generator=gen, device=DEV))
        mid = torch.randn(pages, Hkv, d, generator=gen, device=DEV) * channel
        half = (1.5 + 0.3 * torch.randn(pages, Hkv, d, generator=gen, device=DEV)).abs() * channel
        both = torch.stack([mid + half, mid - half], dim=2)
        codes, s["k_scale"] = _quantise(both)
        v = codes.float() / 4
        s["k_bounds"] = torch.stack([torch.ceil(v[:, :, 0]), torch.floor(v[:, :, 1])], dim=2).to(torch.int8)
    else:
        s["k_cache"], s["k_scale"] = _cache(gen, pages, Hkv, ps, d, 0.5)
        s["v_cache"], s["v_scale"] = _cache(gen, pages, Hkv, ps, d, 0.2)
    if op == "read":
        s["cu"] = i32([0] + np.cumsum(old).tolist())
        s["total"] = sum(old)
        return s
    s.update(scale=1.0 / math.sqrt(d), chosen=c["chosen"], Hkv=Hkv)
    q = 1.5 * torch.randn(B, c["Hq"], c["Sq"], d, generator=gen, device=DEV)
    s["q"] = q.to(torch.bfloat16)
    if op == "decode" and c["chosen"]:
        # lists as a selection gives them: the first and the last block and others, ascending
        n = torch.tensor([_pages(x, ps) for x in old], device=DEV)
        key = torch.rand(B, Hkv, room, generator=gen, device=DEV)
        blk = torch.arange(room, device=DEV)
        key = torch.where((blk == 0) | (blk == n[:, None, None] - 1), torch.full_like(key, 2.0), key)
        key = torch.where(blk < n[:, None, None], key, torch.full_like(key, -1.0))
        take = min(c["chosen"], room)
        best, idx = key.topk(take, dim=2)
        idx = torch.where(best >= 0, idx, room).sort(dim=2).values
        sel = torch.full((B, Hkv, c["chosen"]), -1, dtype=torch.int32, device=DEV)
        sel[:, :, :take] = torch.where(idx < room, idx, -1).int()
        s["sel"], s["n_sel"] = sel, (sel >= 0).sum(dim=2).int()
    return s


# ------------------------------------------------------------ plain forms --

def _plain_assign(s):
    ps, table, free = s["ps"], s["table"], s["free"]
    B, room = table.shape
    seq, new = s["seqlens"].long().clamp(min=0), s["newlens"].long().clamp(min=0)
    have, full = (seq + ps - 1) // ps, (seq + new + ps - 1) // ps
    cu_new = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    never = (full > room) | (cu_new[1:] > s["total"])
    need = torch.where(never, 0, full - have)
    end = need.cumsum(0)
    start = end - need
    refused = never | ((need > 0) & (end > free.numel()))
    used = torch.where(refused | (need == 0), 0, end).amax().reshape(1)
    blk = torch.arange(room, device=DEV)
    fresh = (~refused[:, None]) & (blk >= have[:, None]) & (blk < full[:, None])
    src = (start[:, None] + blk - have[:, None]).clamp(0, max(free.numel() - 1, 0))
    table.copy_(torch.where(fresh, free[src] if free.numel() else table, table))
    t = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(cu_new, t, right=True) - 1
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = seq[b] + t - cu_new[b]
    page = table[b, (pos // ps).clamp(max=room - 1)].long()
    slots = torch.where(inside & ~refused[b] & (page >= 0), page * ps + pos % ps, -1)
    out = torch.where(refused, seq, seq + new)
    cu_k = torch.nn.functional.pad(out.cumsum(0), (1, 0))
    return dict(table=table, slots=slots, cu_new=cu_new.int(), seqlens=out.int(), cu_k=cu_k.int(), used=used.int())


def _plain_store(x, pages, inv, off, n_old, cache, scale, bounds):
    """One of K and V [Hkv, n, d] into its cache; pages are the touched pages, inv each token's of them."""
    x = x.float().transpose(0, 1)  # [n, Hkv, d]
    P, ps = pages.numel(), cache.shape[2]
    fin = torch.where(torch.isfinite(x), x.abs(), 0)
    top = torch.zeros(P, x.shape[1], device=DEV).scatter_reduce_(0, inv[:, None].expand(-1, x.shape[1]),
                                                                 fin.amax(dim=2), "amax")
    m, ex = torch.frexp(top)
    tok = _pow2((ex - 9 + (m > 0.875).int()).clamp(-100, 119))
    kept = n_old[:, None] > 0
    was = torch.where(kept, scale[pages], tok)
    now = torch.maximum(was, tok)
    ratio = was / now
    held = cache[pages].view(torch.uint8).view(F8).float()
    again = (held * ratio[:, :, None, None]).clamp(-448, 448).to(F8)
    keep = (torch.arange(ps, device=DEV) < n_old[:, None])[:, None, :, None]
    codes = cache.view(torch.uint8)
    codes[pages] = torch.where(keep, again.view(torch.uint8), codes[pages])
    y = (x / now[inv][:, :, None]).clamp(-448, 448).to(F8)
    codes[pages[inv], :, off] = y.view(torch.uint8)
    scale[pages] = now
    if bounds is not None:
        v = torch.nan_to_num(y.float()) / 4
        grow = kept[:, :, None]
        o = bounds[pages].float()
        hi = torch.where(grow, torch.ceil(o[:, :, 0] * ratio[:, :, None]), -128.0)
        lo = torch.where(grow, torch.floor(o[:, :, 1] * ratio[:, :, None]), 127.0)
        at = inv[:, None, None].expand_as(v)
        hi = hi.scatter_reduce(0, at, torch.ceil(v), "amax")
        lo = lo.scatter_reduce(0, at, torch.floor(v), "amin")
        bounds[pages] = torch.stack([hi, lo], dim=2).to(torch.int8)


def _plain_write(s):
    ps = s["ps"]
    page, off = s["slots"] // ps, s["slots"] % ps
    pages, inv = torch.unique(page, return_inverse=True)
    n_old = torch.full((pages.numel(),), ps, device=DEV).scatter_reduce_(0, inv, off, "amin")
    _plain_store(s["k"], pages, inv, off, n_old, s["k_cache"], s["k_scale"], s["k_bounds"])
    _plain_store(s["v"], pages, inv, off, n_old, s["v_cache"], s["v_scale"], None)
    return _written(s)


def _written(s):
    out = dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["k_bounds"] is not None:
        out["k_bounds"] = s["k_bounds"]
    return out


def _plain_decode(s):
    q, table, ps = s["q"], s["table"], s["ps"]
    B, Hq, Sq, d = q.shape
    Hkv, room = s["Hkv"], table.shape[1]
    n = s["seqlens"].long()
    if s["chosen"]:
        blk = s["sel"].long()
    else:
        blk = torch.arange(room, device=DEV).expand(B, Hkv, room)
    pos = blk[..., None] * ps + torch.arange(ps, device=DEV)
    page = table[torch.arange(B, device=DEV)[:, None, None], blk.clamp(min=0)].long().clamp(min=0)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    k = s["k_cache"].view(torch.uint8)[page, head].view(F8).float()
    k = (k * s["k_scale"][page, head][..., None, None]).reshape(B, Hkv, -1, d)
    x = (q.float().reshape(B, Hkv, -1, d) @ k.transpose(2, 3)) * s["scale"]
    del k
    last = n[:, None] - Sq + torch.arange(Sq, device=DEV)  # the last key that query row i sees
    last = last.repeat(1, Hq // Hkv)[:, None, :, None]
    at = pos.reshape(B, Hkv, 1, -1)
    x = torch.where((at >= 0) & (at <= last), x, -math.inf)
    top = x.amax(dim=3, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, 0))
    total = e.sum(dim=3, keepdim=True)
    v = s["v_cache"].view(torch.uint8)[page, head].view(F8).float()
    v = (v * s["v_scale"][page, head][..., None, None]).reshape(B, Hkv, -1, d)
    o = (e @ v) / torch.where(total > 0, total, 1)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return dict(o=o.reshape(B, Hq, Sq, d).to(torch.bfloat16), lse=lse.reshape(B, Hq, Sq))


def _plain_select(s):
    q, table, ps = s["q"], s["table"], s["ps"]
    B, Hq, Sq, d = q.shape
    Hkv, room, want = s["Hkv"], table.shape[1], s["chosen"]
    n = ((s["seqlens"].long() + ps - 1) // ps)[:, None, None]
    rows = q.float().reshape(B, Hkv, -1, d)
    m, ex = torch.frexp(rows.abs().amax(dim=3))
    e = (ex - 7 + (m > 127 / 128).int()).clamp(-100, 119)
    q8 = torch.round(rows * _pow2(-e)[..., None])
    page = table.long().clamp(min=0)
    b = s["k_bounds"][page].float().permute(0, 2, 3, 4, 1)  # [B, Hkv, 2, d, blocks]
    u = q8.clamp(min=0) @ b[:, :, 0] + q8.clamp(max=0) @ b[:, :, 1]
    scores = (u * s["k_scale"][page].transpose(1, 2)[:, :, None] * _pow2(e + 2)[..., None]).amax(dim=2)
    blk = torch.arange(room, device=DEV)
    scores = torch.where((blk < 1) | (blk >= n - 1), math.inf, scores)
    scores = torch.where(blk < n, scores, -math.inf)
    best, idx = scores.sort(dim=2, descending=True, stable=True)
    live = torch.arange(room, device=DEV) < torch.minimum(n, torch.tensor(want, device=DEV))
    idx = torch.where(live, idx, room)[:, :, :want].sort(dim=2).values
    sel = torch.full((B, Hkv, want), -1, dtype=torch.int32, device=DEV)
    sel[:, :, :idx.shape[2]] = torch.where(idx < room, idx, -1).int()
    return dict(sel=sel, n_sel=(sel >= 0).sum(dim=2).int())


def _plain_read(s):
    ps = s["ps"]
    t = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    pos = t - s["cu"][b]
    page = s["table"][b, pos // ps].long()

    def one(cache, scale):
        x = cache.view(torch.uint8)[page, :, pos % ps].view(F8).float() * scale[page][..., None]
        return x.transpose(0, 1).to(torch.bfloat16).contiguous()

    return dict(k=one(s["k_cache"], s["k_scale"]), v=one(s["v_cache"], s["v_scale"]))


# ------------------------------------------------------- the framework's --

def _own(s):
    import io_aware_exact_tcgen05_gb300 as fa
    op = s["op"]
    if op == "assign":
        slots, cu_new, seqlens, cu_k, used = fa.fa_kv_assign(s["seqlens"], s["newlens"], s["ps"], s["table"],
                                                             s["free"], s["total"])
        return dict(table=s["table"], slots=slots, cu_new=cu_new, seqlens=seqlens, cu_k=cu_k, used=used)
    if op == "write":
        fa.fa_kv_write_fp8(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                           k_bounds=s["k_bounds"])
        return _written(s)
    if op == "decode":
        o, lse = fa.fa_decode_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                        s["seqlens"], s["scale"], sel=s.get("sel"), n_sel=s.get("n_sel"))
        return dict(o=o, lse=lse)
    if op == "select":
        sel, n_sel = fa.fa_select_blocks(s["q"], s["k_bounds"], s["k_scale"], s["table"], s["seqlens"], s["ps"],
                                         s["chosen"], n_first=1, n_last=1)
        return dict(sel=sel, n_sel=n_sel)
    k, v = fa.fa_kv_read_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["cu"], s["total"])
    return dict(k=k, v=v)


def run(state):
    if own:
        return _own(state)
    return dict(assign=_plain_assign, write=_plain_write, decode=_plain_decode, select=_plain_select,
                read=_plain_read)[state["op"]](state)


def work(case):
    c = case
    old, new = _len_lists(c)
    ps, B, op = c["page"], c["B"], c["op"]
    n_new = sum(new)
    grown = sum(_pages(a + b, ps) - _pages(a, ps) for a, b in zip(old, new))
    if op == "assign":
        # lengths in; slots, offsets and lengths out; each new page moved from the free list to the table
        return {"bytes": 8 * B + 8 * n_new + 4 * (3 * B + 3) + 8 * grown, "flops": 0}
    Hkv, d = c["Hkv"], c["d"]
    if op == "write":
        touched = sum(_pages(a + b, ps) - a // ps for a, b in zip(old, new) if b)
        per_page = 2 * (4 + 4) + (4 * d if c["bounds"] else 0)
        return {"bytes": 2 * n_new * Hkv * d * 3 + 8 * n_new + touched * Hkv * per_page, "flops": 4 * n_new * Hkv * d}
    if op == "read":
        n = sum(old)
        pages = sum(_pages(x, ps) for x in old)
        return {"bytes": 2 * n * Hkv * d * 3 + pages * (8 * Hkv + 4), "flops": 2 * n * Hkv * d}
    rows = c["Hq"] * c["Sq"]
    if op == "select":
        pages = sum(_pages(x, ps) for x in old)
        return {"bytes": pages * (Hkv * (2 * d + 4) + 4) + 2 * B * rows * d + 4 * B * Hkv * (c["chosen"] + 1),
                "flops": 4 * pages * rows * d}
    keys, pages = 0, 0
    for x in old:
        n = _pages(x, ps)
        if c["chosen"] and c["chosen"] < n:
            n = c["chosen"]
            keys += (n - 1) * ps + x - (_pages(x, ps) - 1) * ps
        else:
            keys += x
        pages += n
    listed_bytes = 4 * B * Hkv * (c["chosen"] + 1) if c["chosen"] else 0
    return {"bytes": 2 * keys * Hkv * d + pages * (8 * Hkv + 4) + 4 * B * rows * d + 4 * B * rows + listed_bytes,
            "flops": 4 * keys * rows * d}


# ---------------------------------------------------------------- 64 bits --

_E4M3 = None


def _values(codes):
    """e4m3 codes as 64-bit values, by the format's definition (bias 7, 3 mantissa bits, 0x7f NaN)."""
    global _E4M3
    if _E4M3 is None:
        t = []
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            v = math.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            t.append(-v if c & 128 else v)
        _E4M3 = torch.tensor(t, dtype=torch.float64)
    return _E4M3.to(codes.device)[codes.view(torch.uint8).long()]


def _exponent(x):
    """The smallest whole e with x <= 2^e."""
    m, ex = torch.frexp(x)
    return ex - (m == 0.5).int()


def _nearest(x):
    """64-bit values to the nearest e4m3 value, ties to the even mantissa, at most 448."""
    a = x.abs()
    step = ((torch.frexp(a.clamp(min=2.0 ** -6))[1].long() + (1023 - 4)) << 52).view(torch.float64)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_assign(s):
    ps, total = s["ps"], s["total"]
    seq, new = s["seqlens"].tolist(), s["newlens"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    slots, at, asked, used, out, cu = np.full(total, -1, np.int64), 0, 0, 0, [], [0]
    for b, (n, m) in enumerate(zip(seq, new)):
        first, last = -(-n // ps), -(-(n + m) // ps)
        fits = last <= table.shape[1] and at + m <= total
        if fits:
            asked += last - first
        if fits and (last == first or asked <= len(free)):
            for j in range(first, last):
                table[b, j] = free[asked - last + j]
                used = asked
            p = np.arange(n, n + m)
            slots[at:at + m] = table[b, p // ps].astype(np.int64) * ps + p % ps
            out.append(n + m)
        else:
            out.append(n)
        at += m
        cu.append(at)
    return dict(table=torch.from_numpy(table), slots=torch.from_numpy(slots), cu_new=torch.tensor(cu),
                seqlens=torch.tensor(out), cu_k=torch.tensor([0] + np.cumsum(out).tolist()), used=torch.tensor([used]))


def _exact_write(s):
    ps, slots = s["ps"], s["slots"].tolist()
    out = {}
    runs, i = [], 0
    while i < len(slots):  # stretches of tokens in one page
        j = i + 1
        while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % ps:
            j += 1
        runs.append((i, j, slots[i] // ps, slots[i] % ps))
        i = j
    if len(runs) > 3000:
        return None
    for name in ("k", "v"):
        codes = _values(s[name + "_cache"])
        scale = s[name + "_scale"].double()
        x = s[name].double()
        bounds = s["k_bounds"].double() if name == "k" and s["k_bounds"] is not None else None
        for i, j, page, off in runs:
            y = x[:, i:j]
            top = y.abs().amax(dim=(1, 2))
            e = torch.where(top > 0, _exponent(top / 448), -100).clamp(-100, 119)
            tok = ((e.long() + 1023) << 52).view(torch.float64)
            was = scale[page] if off else tok
            now = torch.maximum(was, tok)
            r = (was / now)[:, None]
            if off:
                codes[page, :, :off] = _nearest(codes[page, :, :off] * r[:, None])
            z = _nearest(y / now[:, None, None])
            codes[page, :, off:off + j - i] = z
            scale[page] = now
            if bounds is not None:
                hi, lo = torch.ceil(z.amax(dim=1) / 4), torch.floor(z.amin(dim=1) / 4)
                if off:
                    hi = torch.maximum(hi, torch.ceil(bounds[page, :, 0] * r))
                    lo = torch.minimum(lo, torch.floor(bounds[page, :, 1] * r))
                bounds[page, :, 0], bounds[page, :, 1] = hi, lo
        out[name], out[name + "_scale"] = codes, scale
        if bounds is not None:
            out["k_bounds"] = bounds.to(torch.int8)
    return out


def _exact_decode(s):
    q, ps, Hkv = s["q"].double(), s["ps"], s["Hkv"]
    B, Hq, Sq, d = q.shape
    G = Hq // Hkv
    o, lse = torch.zeros_like(q), torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seqlens"].tolist()):
        for h in range(Hkv):
            if s["chosen"]:
                blk = s["sel"][b, h, :int(s["n_sel"][b, h])].long()
            else:
                blk = torch.arange(_pages(n, ps), device=DEV)
            page = s["table"][b, blk].long()
            pos = (blk[:, None] * ps + torch.arange(ps, device=DEV)).reshape(-1)
            live = pos < n
            pos = pos[live]
            k = (_values(s["k_cache"][page, h]) * s["k_scale"][page, h].double()[:, None, None]).reshape(-1, d)[live]
            v = (_values(s["v_cache"][page, h]) * s["v_scale"][page, h].double()[:, None, None]).reshape(-1, d)[live]
            x = torch.einsum("gid,kd->gik", q[b, h * G:(h + 1) * G], k) / math.sqrt(d)
            seen = pos[None, :] <= (n - Sq + torch.arange(Sq, device=DEV))[:, None]
            x = x.masked_fill(~seen, -math.inf)
            w = torch.nan_to_num(torch.softmax(x, dim=2)) * seen
            o[b, h * G:(h + 1) * G] = torch.einsum("gik,kd->gid", w, v)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=2)
    return dict(o=o, lse=lse)


def _exact_select(s):
    q, ps, Hkv, want = s["q"].double().cpu().numpy(), s["ps"], s["Hkv"], s["chosen"]
    B, Hq, Sq, d = q.shape
    table, lens = s["table"].cpu().numpy(), s["seqlens"].tolist()
    bounds, scale = s["k_bounds"].cpu().numpy().astype(np.int64), s["k_scale"].double().cpu().numpy()
    sel = np.full((B, Hkv, want), -1, np.int64)
    for b in range(B):
        n = _pages(lens[b], ps)
        page = table[b, :n]
        for h in range(Hkv):
            rows = q[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].reshape(-1, d)
            best = np.full(n, -np.inf)
            for row in rows:
                top = np.abs(row).max()
                m, e = math.frexp(top / 127)
                e = max(-100, min(119, e - (m == 0.5))) if top > 0 else -100
                w = np.rint(row / 2.0 ** e).astype(np.int64)
                u = np.maximum(w * bounds[page, h, 0], w * bounds[page, h, 1]).sum(axis=1)
                best = np.maximum(best, u * scale[page, h] * 2.0 ** (e + 2))
            best[:1] = np.inf
            best[n - 1:] = np.inf
            got = np.sort(np.argsort(-best, kind="stable")[:want])
            sel[b, h, :len(got)] = got
    return dict(sel=torch.from_numpy(sel), n_sel=torch.from_numpy((sel >= 0).sum(axis=2)))


def _exact_read(s):
    out = {}
    for name in ("k", "v"):
        rows = []
        for b, n in enumerate((s["cu"][1:] - s["cu"][:-1]).tolist()):
            page = s["table"][b, :_pages(n, s["ps"])].long()
            x = _values(s[name + "_cache"][page]) * s[name + "_scale"][page].double()[:, :, None, None]
            rows.append(x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n])
        out[name] = torch.cat(rows, dim=1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(assign=_exact_assign, write=_exact_write, decode=_exact_decode, select=_exact_select,
                read=_exact_read)[s["op"]](s)
