"""GPU tests of the paged 8-bit KV cache operators against their plain 64-bit
definitions (oracle/paged.py).  Integers, codes, scales and bounds have to be
equal; attention is held to element-wise rounding bounds (tests/paged.py)."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import paged as po
from tests.paged import (DEV, check_attention, f64, i32, make_cache, make_table, on_gpu,
                         randn_bf16)

pytestmark = pytest.mark.gpu

SENT = 0x5b  # byte that untouched memory keeps


# ----------------------------------------------------------------- assign --

def _check_assign(seq, new, ps, room, n_free, total, seed=0, table=None):
    rng = np.random.RandomState(seed)
    pool = rng.permutation(n_free + 4 * len(seq) * room)
    free = pool[:n_free]
    if table is None:
        table = np.full((len(seq), room), -7, np.int64)
        at = n_free
        for b, n in enumerate(seq):
            m = min(po.pages_of(max(n, 0), ps), room)
            table[b, :m] = pool[at:at + m]
            at += m
    want = po.assign(seq, new, ps, table, free, total)
    t = i32(table)
    slots, cu, out, cuk, used = fa.fa_kv_assign(i32(seq), i32(new), ps, t, i32(free), total)
    torch.cuda.synchronize()
    for name, got, ref in (("table", t, want[0]), ("slots", slots, want[1]), ("cu_new", cu, want[2]),
                           ("seqlens_out", out, want[3]), ("cu_k", cuk, want[4])):
        assert np.array_equal(got.cpu().numpy().astype(np.int64), ref), name
    assert int(used) == want[5]
    return want


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 31, 255, 256, 257, 600])
def test_assign_step_and_prompts(ps, B):
    rng = np.random.RandomState(B + ps)
    seq = rng.randint(0, 300, B)
    _check_assign(seq, np.ones(B, int), ps, 30, B, B, seed=1)
    new = rng.randint(0, 70, B)
    _check_assign(seq, new, ps, 30, 6 * B, int(new.sum()), seed=2)


def test_assign_long_prompts_and_padding():
    # many CTAs' worth of tokens, and packed rows behind the last request
    _check_assign([0, 17, 5000], [9000, 1, 4097], 16, 700, 2000, 9000 + 1 + 4097 + 77)
    _check_assign([3], [0], 16, 2, 0, 5)          # nothing to place
    _check_assign([16, 32], [0, 0], 16, 2, 0, 0)  # no packed rows at all


def test_assign_refusals_leave_the_request_as_it_was():
    # too few free pages (and those behind it), too many blocks, too many tokens
    want = _check_assign([10, 20, 30, 5], [30, 100, 1, 40], 16, 10, 6, 171)
    assert list(want[3]) == [40, 20, 31, 5]
    want = _check_assign([10, 150, 30], [30, 20, 10], 16, 10, 20, 60)
    assert list(want[3]) == [40, 150, 40]
    want = _check_assign([10, 20, 30], [30, 20, 10], 16, 10, 20, 55)
    assert list(want[3]) == [40, 40, 30]
    # negative lengths count as 0; a length past the table is refused
    want = _check_assign([-5, 1000], [4, 1], 16, 4, 9, 5)
    assert list(want[3]) == [4, 1000]


def test_assign_absent_page_gives_no_slot():
    table = np.array([[5, -1, -1], [6, -1, -1]])
    want = _check_assign([20, 3], [2, 2], 16, 3, 4, 4, table=table)
    assert list(want[1][:2]) == [-1, -1] and want[1][2] == 6 * 16 + 3


# ------------------------------------------------------------------ write --

def _write_and_check(cache, k, v, slots, bounds=True, token_major=False):
    """k, v bf16 CPU [Hkv, n, d] into the oracle's cache and a copy on the GPU."""
    kc, vc, ks, vs, kb = on_gpu(cache)
    if token_major:
        both = torch.stack([k, v], 2).permute(1, 2, 0, 3).contiguous().to(DEV)  # [n, 2, H, d]
        gk, gv = both[:, 0].transpose(0, 1), both[:, 1].transpose(0, 1)
    else:
        gk, gv = k.to(DEV), v.to(DEV)
    if not bounds:
        cache.bounds = None
    cache.write(f64(k), f64(v), slots)
    fa.fa_kv_write_fp8(gk, gv, torch.tensor(slots, dtype=torch.int64, device=DEV), kc, vc, ks, vs,
                       k_bounds=kb if bounds else None)
    torch.cuda.synchronize()
    # NaN codes may carry either sign
    for got, ref, name in ((kc, cache.codes[0], "k"), (vc, cache.codes[1], "v")):
        got = got.cpu().numpy()
        nan = (ref & 127) == 127
        assert np.array_equal((got & 127) == 127, nan), f"{name} NaN codes"
        assert np.array_equal(got[~nan], ref[~nan]), f"{name} codes"
    assert np.array_equal(f64(ks), cache.scale[0]) and np.array_equal(f64(vs), cache.scale[1])
    if bounds:
        assert np.array_equal(kb.cpu().numpy().astype(np.int64), cache.bounds)
    return kc, vc, ks, vs, kb


def _slots_of(table, starts, counts, ps):
    out = []
    for b, (s, n) in enumerate(zip(starts, counts)):
        out += [int(table[b, (s + i) // ps]) * ps + (s + i) % ps for i in range(n)]
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("token_major", [False, True])
def test_write_runs(d, ps, token_major):
    gen = torch.Generator().manual_seed(ps + d)
    starts, counts = [0, 1, ps - 1, ps, 2 * ps + 3, 5, 0], [1, ps, 2, 3 * ps + 1, 1, 0, 2 * ps]
    pages = sum(po.pages_of(s + n, ps) for s, n in zip(starts, counts))
    table = make_table(3, [s + n for s, n in zip(starts, counts)], ps, pages)
    n = sum(counts)
    # louder and quieter than what the pages hold, so that some scales grow
    k = randn_bf16(gen, 3, n, d, mult=1.5) * torch.exp2(torch.randint(-3, 4, (3, n, 1), generator=gen))
    v = randn_bf16(gen, 3, n, d, mult=1.5)
    _write_and_check(make_cache(ps, pages, 3, ps, d), k.to(torch.bfloat16), v,
                     _slots_of(table, starts, counts, ps), token_major=token_major)


def test_write_steps_keep_a_page_consistent():
    # 40 single tokens into the same pages, one call each, growing in size
    ps, d = 16, 64
    cache = make_cache(5, 4, 2, ps, d)
    dev = on_gpu(cache)
    gen = torch.Generator().manual_seed(8)
    for t in range(40):
        k = randn_bf16(gen, 2, 2, d, mult=2.0 ** (t // 5 - 3))
        v = randn_bf16(gen, 2, 2, d, mult=2.0 ** -(t // 3))
        slots = [(t // ps) * ps + t % ps, 3 * ps + t % ps]
        cache.write(f64(k), f64(v), slots)
        fa.fa_kv_write_fp8(k.to(DEV), v.to(DEV), torch.tensor(slots, device=DEV), *dev[:4],
                           k_bounds=dev[4])
    for got, ref in zip(dev, cache.codes + cache.scale + [cache.bounds]):
        assert np.array_equal(f64(got), np.asarray(ref, np.float64))


def test_write_special_values():
    ps, d = 32, 128
    gen = torch.Generator().manual_seed(4)
    k, v = randn_bf16(gen, 2, 40, d), randn_bf16(gen, 2, 40, d)
    k[0, 3, 5], k[0, 4, 6], k[1, 2, 7] = math.inf, -math.inf, math.nan
    v[:, 8:40] = 0.0                      # a run of zeros only
    v[0, 1] = math.nan                    # a token of NaN only
    k[1, 33:] = 3.3e38                    # past the largest scale: saturates
    k[1, 32] = 1e-38
    _write_and_check(make_cache(6, 4, 2, ps, d), k, v, list(range(ps, ps + 40)))
    tiny = torch.full((2, 3, d), 1e-39).to(torch.bfloat16)
    _write_and_check(make_cache(7, 4, 2, ps, d), tiny, tiny * 0, [0, 1, 2])


def test_write_keeps_a_scale_that_is_no_power_of_two():
    ps, d = 16, 64
    cache = make_cache(9, 3, 2, ps, d)
    cache.scale = [np.float32(s * 1.3).astype(np.float64) for s in cache.scale]
    kc = [c.copy() for c in cache.codes]
    gen = torch.Generator().manual_seed(5)
    k, v = randn_bf16(gen, 2, 5, d, mult=0.5), randn_bf16(gen, 2, 5, d, mult=9.0)
    ref = po.Cache(*kc, *cache.scale, cache.bounds)
    dev = on_gpu(cache)
    slots = [3, 4, 5, ps + 1, ps + 2]
    fa.fa_kv_write_fp8(k.to(DEV), v.to(DEV), torch.tensor(slots, device=DEV), *dev[:4],
                       k_bounds=dev[4])
    ref.write(f64(k), f64(v), slots)
    assert np.array_equal(f64(dev[2]), ref.scale[0]) and np.array_equal(f64(dev[3]), ref.scale[1])
    # The quotient is formed in fp32 before it is rounded to e4m3.  Its error is at most 2^-24 of
    # it, so a code can differ from the one of the 64-bit quotient only where that quotient lies
    # within 2^-24 of the midpoint between the two codes (1.3 * 25 / 16 is nearly a bf16 value,
    # so such quotients are met); a held code's ratio adds one more rounding.
    for which, x in ((0, f64(k)), (1, f64(v))):
        exact = po.decode_codes(kc[which])
        for page, off, lo, n in ((0, 3, 0, 3), (1, 1, 3, 2)):
            now = ref.scale[which][page][:, None, None]
            exact[page, :, :off] *= np.asarray(cache.scale[which][page])[:, None, None] / now
            exact[page, :, off:off + n] = x[:, lo:lo + n] / now
        got = dev[which].cpu().numpy()
        differ = got != ref.codes[which]
        mid = (po.decode_codes(got[differ]) + po.decode_codes(ref.codes[which][differ])) / 2
        assert np.all(np.abs(exact[differ] - mid) <= 2 * 2.0 ** -24 * np.abs(mid))


def test_write_skips_slots_outside_the_cache_and_touches_nothing_else():
    ps, d, pages = 16, 64, 5
    cache = make_cache(11, pages, 2, ps, d)
    gen = torch.Generator().manual_seed(6)
    slots = [-1, -5, pages * ps, 2 ** 40, 33, 34, -1, 3, 79, pages * ps + 3]
    k, v = randn_bf16(gen, 2, len(slots), d), randn_bf16(gen, 2, len(slots), d)
    _write_and_check(cache, k, v, slots)
    _write_and_check(make_cache(12, pages, 2, ps, d), k, v, slots, bounds=False)


def test_write_many_tokens_and_a_rolled_back_page():
    # more tokens than one launch shape covers; then a page is written again from its middle
    ps, d = 64, 128
    gen = torch.Generator().manual_seed(13)
    n = 3000
    pages = n // ps + 2
    cache = make_cache(14, pages, 1, ps, d)
    order = np.random.RandomState(2).permutation(pages)
    slots = [int(order[(7 + i) // ps]) * ps + (7 + i) % ps for i in range(n)]
    _write_and_check(cache, randn_bf16(gen, 1, n, d), randn_bf16(gen, 1, n, d), slots)
    back = [int(order[3]) * ps + 20 + i for i in range(9)]
    _write_and_check(cache, randn_bf16(gen, 1, 9, d, mult=4.0), randn_bf16(gen, 1, 9, d), back)


# ------------------------------------------------------------------- read --

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 128])
def test_read_ragged(d, ps):
    lens = [0, 1, ps, 3 * ps + 5, 0, 17]
    pages = sum(po.pages_of(n, ps) for n in lens) + 1
    cache = make_cache(d + ps, pages, 2, ps, d)
    table = make_table(4, lens, ps, pages, room=5)
    table[3, 1] = pages + 3  # a block without a page reads as zeros
    cu = np.cumsum([0] + lens)
    total = int(cu[-1]) + 6
    k = torch.full((2, total, d), 7.0, dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, 7.0)
    kc, vc, ks, vs, _ = on_gpu(cache)
    fa.fa_kv_read_fp8(kc, vc, ks, vs, i32(table), i32(cu), total, k=k, v=v)
    torch.cuda.synchronize()
    for which, got in ((0, f64(k)), (1, f64(v))):
        for s, n in enumerate(lens):
            for h in range(2):
                ref, _ = cache.gather(which, table[s], h, np.arange(n))
                assert np.array_equal(got[h, cu[s]:cu[s + 1]], ref)  # 4 bits times a power of two
        assert np.all(got[:, int(cu[-1]):] == 7.0), "rows of no sequence"


def test_read_past_the_table_gives_zeros_and_empty_reads():
    cache = make_cache(1, 3, 1, 16, 64)
    kc, vc, ks, vs, _ = on_gpu(cache)
    table = i32([[2, 0]])
    k, v = fa.fa_kv_read_fp8(kc, vc, ks, vs, table, i32([0, 40]), 40)
    assert np.all(f64(k)[:, 32:] == 0) and np.all(f64(v)[:, 32:] == 0)
    assert np.array_equal(f64(k)[0, :16], cache.values(0, 2, 0))
    k, v = fa.fa_kv_read_fp8(kc, vc, ks, vs, table, i32([0, 0]), 0)
    assert k.shape == (1, 0, 64)


# ----------------------------------------------------------------- select --

def _select_case(B, Hq, heads, Sq, d, ps, lens, k, first=1, last=1, seed=0, room=None, hide=()):
    room = room or max(1, max(po.pages_of(max(n, 0), ps) for n in lens))
    pages = sum(po.pages_of(max(n, 0), ps) for n in lens) + 2
    rng = np.random.RandomState(seed)
    mid = rng.randint(-80, 80, (pages, heads, 1, d))
    half = rng.randint(0, 32, (pages, heads, 1, d))
    bounds = np.concatenate([mid + half, mid - half], axis=2)
    scale = 2.0 ** rng.randint(-9, -5, (pages, heads))
    table = make_table(seed, lens, ps, pages, room=room)
    for b, i in hide:
        table[b, i] = -1
    q = randn_bf16(torch.Generator().manual_seed(seed), B, Hq, Sq, d, mult=3.0)
    want = po.select(f64(q), bounds, scale, table, lens, ps, k, first, last)
    sel, n_sel = fa.fa_select_blocks(
        q.to(DEV), torch.from_numpy(bounds.astype(np.int8)).to(DEV),
        torch.from_numpy(scale.astype(np.float32)).to(DEV), i32(table), i32(lens), ps, k,
        n_first=first, n_last=last)
    torch.cuda.synchronize()
    assert np.array_equal(n_sel.cpu().numpy(), want[1])
    assert np.array_equal(sel.cpu().numpy(), want[0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", [(1, 1, 1), (8, 2, 1), (6, 2, 3), (32, 1, 2)])
def test_select_groups(d, Hq, heads, Sq):
    _select_case(3, Hq, heads, Sq, d, 16, [16 * 37, 500, 33], 9, seed=d + Hq)


@pytest.mark.parametrize("k,first,last", [(1, 0, 0), (1, 1, 0), (5, 2, 3), (64, 1, 1), (300, 0, 2)])
def test_select_counts(k, first, last):
    lens = [0, 1, 64, 65, 64 * 63, 64 * 64 + 1, 64 * 200, 30]
    _select_case(len(lens), 4, 2, 1, 64, 64, lens, k, first, last, seed=k)


def test_select_long_and_hidden_blocks():
    _select_case(2, 4, 1, 1, 128, 16, [16 * 5001 - 3, 16 * 900], 128, seed=3,
                 hide=[(0, 7), (0, 4000), (1, 899)])
    # fewer blocks with a page than asked for: the absent ones rank last, by index
    _select_case(1, 2, 1, 1, 64, 16, [16 * 8], 6, first=0, last=0, seed=5,
                 hide=[(0, i) for i in (1, 2, 3, 6, 7)])
    # lengths behind the table and below zero are clamped
    _select_case(2, 2, 1, 1, 64, 16, [16 * 4, -3], 3, seed=6, room=4)


def test_select_ties_take_the_lower_block():
    q = torch.ones(1, 2, 1, 64, dtype=torch.bfloat16, device=DEV)
    bounds = torch.ones(40, 1, 2, 64, dtype=torch.int8, device=DEV)
    scale = torch.ones(40, 1, device=DEV)
    scale[30] = 2.0
    table = torch.arange(40, dtype=torch.int32, device=DEV).reshape(1, 40)
    sel, n = fa.fa_select_blocks(q, bounds, scale, table, i32([640]), 16, 6, n_first=0, n_last=1)
    assert sel.cpu().tolist() == [[[0, 1, 2, 3, 30, 39]]] and n.cpu().tolist() == [[6]]
    sel, n = fa.fa_select_blocks(q * 0, bounds, scale, table, i32([640]), 16, 4, n_first=0, n_last=0)
    assert sel.cpu().tolist() == [[[0, 1, 2, 3]]]


# ----------------------------------------------------------------- decode --

def _decode_case(lens, Hq, heads, Sq, d, ps, seed=0, q_mult=1.0, scale=None, sel=None, n_sel=None,
                 room=None, cache=None, table=None):
    pages = sum(po.pages_of(max(n, 0), ps) for n in lens) + 2
    cache = cache or make_cache(seed, pages, heads, ps, d)
    table = make_table(seed + 1, lens, ps, pages, room=room) if table is None else table
    scale = 1 / math.sqrt(d) if scale is None else scale
    q = randn_bf16(torch.Generator().manual_seed(seed + 2), len(lens), Hq, Sq, d, mult=q_mult)
    ref = po.attend(f64(q), cache, table, lens, scale, sel, n_sel)
    kc, vc, ks, vs, _ = on_gpu(cache)
    more = {} if sel is None else dict(sel=i32(sel), n_sel=i32(n_sel))
    o, lse = fa.fa_decode_paged_fp8(q.to(DEV), kc, vc, ks, vs, i32(table), i32(lens), scale, **more)
    torch.cuda.synchronize()
    check_attention(o, lse, ref, max(max(lens), 1), d)
    assert fa.fa_device_status()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", [(1, 1, 1), (4, 4, 1), (8, 2, 1), (9, 3, 2), (16, 1, 1),
                                         (20, 2, 1), (8, 1, 4), (12, 2, 5), (32, 1, 3)])
def test_decode_groups_and_rows(d, Hq, heads, Sq):
    _decode_case([300, 5, 77], Hq, heads, Sq, d, 16, seed=d + Hq + Sq)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 129, 1000])
def test_decode_lengths(ps, n):
    _decode_case([n, 0, max(n // 2, 1), n - 1], 4, 2, 1, 128, ps, seed=n)


def test_decode_long_ragged():
    _decode_case([9001, 40, 2500], 4, 1, 1, 128, 64, seed=1)
    _decode_case([6000], 8, 8, 2, 64, 32, seed=2)


def test_decode_rows_that_see_nothing():
    # more query rows than keys: the first rows see none
    _decode_case([0, 1, 2, 5, 3], 4, 2, 5, 64, 16, seed=3)


def test_decode_many_requests():
    lens = [int(x) for x in np.random.RandomState(0).randint(0, 90, 200)]
    _decode_case(lens, 2, 1, 1, 64, 16, seed=4)
    lens = [int(x) for x in np.random.RandomState(1).randint(0, 20, 700)]
    _decode_case(lens, 2, 2, 1, 64, 16, seed=5)  # 1400 items: several for each thread of the plan
    _decode_case(lens[:300], 18, 2, 1, 64, 16, seed=6)


def test_decode_many_rows():
    # several row blocks of the wide kernel, the last one partial, over a few CTAs' stretches
    _decode_case([700, 31], 24, 2, 11, 64, 32, seed=7)
    _decode_case([150], 32, 1, 5, 128, 64, seed=8)


def test_decode_large_logits_and_zero_scale():
    _decode_case([700, 130], 8, 2, 1, 128, 64, seed=5, q_mult=40.0)
    _decode_case([700, 130], 8, 2, 1, 128, 64, seed=6, scale=0.0)


@pytest.mark.parametrize("mult", [2.0 ** -60, 2.0 ** 50, 2.0 ** 90])
def test_decode_query_sizes(mult):
    _decode_case([200, 3], 4, 2, 1, 64, 16, seed=7, q_mult=mult, scale=0.125 / mult)


def test_decode_one_dominant_key_and_many_light_ones():
    # the light keys' weights are 2^-26 each: together they still count
    ps, d, n = 64, 64, 4096
    cache = make_cache(1, n // ps, 1, ps, d)
    cache.scale = [np.ones_like(s) for s in cache.scale]
    cache.codes[0][:] = 0
    cache.codes[1][:] = po.encode(np.array(1.0))
    table = np.arange(n // ps).reshape(1, -1)
    cache.codes[0][0, 0, 0, 0] = po.encode(np.array(1.0))
    cache.codes[1][0, 0, 0] = 0
    q = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16)
    q[..., 0] = 16.0
    ref = po.attend(f64(q), cache, table, [n], 1.125)
    kc, vc, ks, vs, _ = on_gpu(cache)
    o, lse = fa.fa_decode_paged_fp8(q.to(DEV), kc, vc, ks, vs, i32(table), i32([n]), 1.125)
    check_attention(o, lse, ref, n, d)
    assert abs(f64(o)[0, 0, 0, 5] / ref[0][0, 0, 0, 5] - 1) < 2.0 ** -7


def test_decode_page_scales_far_apart():
    # V scales from 2^-20 to 2^20 and K scales that differ by page, some no powers of two
    ps, d, lens = 16, 64, [200, 130]
    cache = make_cache(8, 30, 2, ps, d)
    rng = np.random.RandomState(3)
    cache.scale[1] = cache.scale[1] * 2.0 ** rng.randint(-20, 21, cache.scale[1].shape)
    cache.scale[0] = np.float32(cache.scale[0] * rng.uniform(0.5, 2, cache.scale[0].shape)).astype(
        np.float64)
    _decode_case(lens, 4, 2, 1, d, ps, seed=9, cache=cache)


def test_decode_ignores_what_lies_behind_the_last_key():
    ps, d, lens = 32, 128, [33, 64, 1]
    cache = make_cache(10, 8, 2, ps, d)
    table = make_table(2, lens, ps, 8)
    for b, n in enumerate(lens):
        for j in range(n, po.pages_of(n, ps) * ps):
            for c in cache.codes:
                c[table[b, j // ps], :, j % ps] = 0x7f  # NaN codes
    _decode_case(lens, 4, 2, 1, d, ps, seed=11, cache=cache, table=table)
    _decode_case(lens, 4, 2, 3, d, ps, seed=12, cache=cache, table=table)


def test_decode_nan_reaches_only_the_rows_that_see_it():
    ps, d, lens = 16, 64, [37, 20]
    for which in (0, 1):
        cache = make_cache(13, 6, 2, ps, d)
        table = make_table(3, lens, ps, 6)
        # the newest key of request 0, head 1: hidden from all rows but the last
        cache.codes[which][table[0, 36 // ps], 1, 36 % ps, 7] = 0x7f
        _decode_case(lens, 4, 2, 4, d, ps, seed=14, cache=cache, table=table)
        # an older key of request 1: every row sees it
        cache.codes[which][table[1, 0], 0, 3, 9] = 0xff
        _decode_case(lens, 4, 2, 4, d, ps, seed=15, cache=cache, table=table)


def test_decode_absent_pages_are_hidden():
    ps, lens = 16, [100, 40]
    cache = make_cache(16, 12, 2, ps, 64)
    table = make_table(4, lens, ps, 12)
    table[0, 2], table[0, 6], table[1, :] = -1, 99, -1
    _decode_case(lens, 4, 2, 1, 64, ps, seed=17, cache=cache, table=table)
    _decode_case([1000, -4], 4, 2, 1, 64, ps, seed=17, cache=cache, table=table)  # clamped lengths


@pytest.mark.parametrize("Sq", [1, 3])
def test_decode_chosen_blocks(Sq):
    ps, lens, heads = 16, [400, 37, 0, 160], 2
    rng = np.random.RandomState(5)
    sel, n_sel = np.full((4, heads, 7), -1), np.zeros((4, heads), int)
    for b, n in enumerate(lens):
        for h in range(heads):
            m = po.pages_of(n, ps)
            take = min(m, rng.randint(0, 8))
            sel[b, h, :take] = np.sort(rng.permutation(m)[:take])
            n_sel[b, h] = take
    _decode_case(lens, 6, heads, Sq, 128, ps, seed=18, sel=sel, n_sel=n_sel)
    # entries outside the request and counts outside the list are ignored; twice counts twice
    sel[0, 0] = [0, 0, 24, 25, -1, 500, 3]
    sel[1, 1] = [2, 1, 0, 9, 9, 9, 9]
    n_sel[0, 0], n_sel[1, 1], n_sel[3, 0] = 7, 50, -2
    _decode_case(lens, 6, heads, Sq, 128, ps, seed=19, sel=sel, n_sel=n_sel)


def test_decode_long_chosen_list():
    ps, n = 16, 16 * 700
    sel = np.sort(np.random.RandomState(1).permutation(700)[:300]).reshape(1, 1, -1)
    _decode_case([n], 4, 1, 1, 64, ps, seed=20, sel=sel, n_sel=np.array([[300]]))


WIDE = [(6, 2, 4, 64), (6, 2, 4, 128), (24, 2, 2, 64), (24, 2, 2, 128), (36, 2, 3, 128)]


@pytest.mark.parametrize("Hq,heads,Sq,d", WIDE)
def test_decode_wide_nan_reaches_only_the_rows_that_see_it(Hq, heads, Sq, d):
    ps, lens = 16, [237, 20]
    for which in (0, 1):
        cache = make_cache(13, 20, heads, ps, d)
        table = make_table(3, lens, ps, 20)
        # the newest key of request 0, head 1: hidden from all rows but the last
        cache.codes[which][table[0, 236 // ps], 1, 236 % ps, 7] = 0x7f
        _decode_case(lens, Hq, heads, Sq, d, ps, seed=34, cache=cache, table=table)
        # the next one, at another channel: hidden from the first rows
        cache.codes[which][table[0, 235 // ps], 1, 235 % ps, d - 1] = 0xff
        _decode_case(lens, Hq, heads, Sq, d, ps, seed=35, cache=cache, table=table)
        # an older key of request 1: every row sees it
        cache.codes[which][table[1, 0], 0, 3, 9] = 0xff
        _decode_case(lens, Hq, heads, Sq, d, ps, seed=36, cache=cache, table=table)


@pytest.mark.parametrize("Hq,heads,Sq,d", WIDE)
def test_decode_wide_absent_pages_and_what_lies_behind_the_last_key(Hq, heads, Sq, d):
    ps, lens = 32, [1500, 33, 40, 64, 1]
    pages = 60
    cache = make_cache(37, pages, heads, ps, d)
    table = make_table(38, lens, ps, pages)
    for b, n in enumerate(lens):
        for j in range(n, po.pages_of(n, ps) * ps):
            for c in cache.codes:
                c[table[b, j // ps], :, j % ps] = 0x7f  # NaN codes
    _decode_case(lens, Hq, heads, Sq, d, ps, seed=39, cache=cache, table=table)
    table[0, [0, 7, 8, 9, 10, 30, 46]] = -1
    table[2, :] = pages  # no page at all: every key is hidden
    _decode_case(lens, Hq, heads, Sq, d, ps, seed=40, cache=cache, table=table)


@pytest.mark.parametrize("Hq,heads,Sq,d", WIDE)
def test_decode_wide_chosen_blocks_and_far_apart_scales(Hq, heads, Sq, d):
    ps, lens = 16, [900, 50, 0]
    cache = make_cache(41, 65, heads, ps, d)
    rng = np.random.RandomState(42)
    cache.scale[1] = cache.scale[1] * 2.0 ** rng.randint(-20, 21, cache.scale[1].shape)
    sel, n_sel = np.full((3, heads, 40), -1), np.zeros((3, heads), int)
    for b, n in enumerate(lens):
        for h in range(heads):
            m = po.pages_of(n, ps)
            take = min(m, rng.randint(1, 41))
            sel[b, h, :take] = np.sort(rng.permutation(m)[:take])
            n_sel[b, h] = take
    table = make_table(43, lens, ps, 65)
    _decode_case(lens, Hq, heads, Sq, d, ps, seed=44, cache=cache, table=table)
    _decode_case(lens, Hq, heads, Sq, d, ps, seed=45, cache=cache, table=table, sel=sel, n_sel=n_sel)
    sel[0, 0, :7] = [0, 0, 56, 57, -1, 500, 3]  # behind the request, absent, twice the same
    n_sel[0, 0], n_sel[1, 1] = 7, 90
    _decode_case(lens, Hq, heads, Sq, d, ps, seed=46, cache=cache, table=table, sel=sel, n_sel=n_sel)


def test_decode_wide_offsets_past_32_bits():
    ps, d, heads = 64, 128, 2
    pages = (1 << 32) // (ps * d * heads) + 64
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    small = make_cache(47, 6, heads, ps, d)
    parts = on_gpu(small)[:4]
    at = torch.tensor([pages - 1, 3, pages - 40, pages - 2, 7, pages - 9], device=DEV)
    big = [torch.empty(pages, *t.shape[1:], dtype=t.dtype, device=DEV) for t in parts]
    for b, t in zip(big, parts):
        b[at] = t
    table = np.array([[0, 1, 2, 3, 4]])
    q = randn_bf16(torch.Generator().manual_seed(1), 1, 40, 1, d)
    o, lse = fa.fa_decode_paged_fp8(q.to(DEV), *big, at[torch.from_numpy(table).to(DEV)].int(),
                                    i32([300]), 0.1)
    check_attention(o, lse, po.attend(f64(q), small, table, [300], 0.1), 300, d)


def test_offsets_past_32_bits():
    # pages of 16 KB: the last ones lie behind 4 GB
    ps, d, heads = 64, 128, 2
    pages = (1 << 32) // (ps * d * heads) + 64
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    small = make_cache(21, 6, heads, ps, d)
    kc, vc, ks, vs, kb = on_gpu(small)
    at = torch.tensor([pages - 1, 3, pages - 40, pages - 2, 7, pages - 9], device=DEV)
    big = [torch.empty(pages, *t.shape[1:], dtype=t.dtype, device=DEV) for t in (kc, vc, ks, vs, kb)]
    for b, t in zip(big, (kc, vc, ks, vs, kb)):
        b[at] = t
    lens, table = [300], np.array([[0, 1, 2, 3, 4]])
    big_table = at[torch.from_numpy(table).to(DEV)].int()
    q = randn_bf16(torch.Generator().manual_seed(1), 1, 4, 1, d)
    o, lse = fa.fa_decode_paged_fp8(q.to(DEV), *big[:4], big_table, i32(lens), 0.1)
    check_attention(o, lse, po.attend(f64(q), small, table, lens, 0.1), 300, d)
    k, v = fa.fa_kv_read_fp8(*big[:4], big_table, i32([0, 300]), 300)
    assert np.array_equal(f64(k)[1], small.gather(0, table[0], 1, np.arange(300))[0])
    # token 300 enters a page behind 4 GB
    x, y = randn_bf16(torch.Generator().manual_seed(2), 2, heads, 1, d)
    page, slot = int(at[4]), int(at[4]) * ps + 300 % ps
    fa.fa_kv_write_fp8(x.to(DEV), y.to(DEV), torch.tensor([slot], device=DEV), *big[:4],
                       k_bounds=big[4])
    small.write(f64(x), f64(y), [4 * ps + 300 % ps])
    assert np.array_equal(big[0][page].cpu().numpy(), small.codes[0][4])
    sel, _ = fa.fa_select_blocks(q.to(DEV), big[4], big[2], big_table, i32([301]), ps, 3)
    want, _ = po.select(f64(q), small.bounds, small.scale[0], table, [301], ps, 3, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)


# ------------------------------------------------------- used as a program --

def test_serving_steps_together():
    """Prompts enter the cache, a prompt chunk attends over its cached prefix, and
    decode steps follow: over every block, and over the chosen ones."""
    heads, Hq, d, ps, room, pages = 2, 8, 64, 16, 40, 90
    scale = 1 / math.sqrt(d)
    gen = torch.Generator().manual_seed(30)
    cache = po.Cache(np.zeros((pages, heads, ps, d), np.uint8),
                     np.zeros((pages, heads, ps, d), np.uint8), np.zeros((pages, heads)),
                     np.zeros((pages, heads)), np.zeros((pages, heads, 2, d)))
    kc, vc, ks, vs, kb = on_gpu(cache)
    free = torch.from_numpy(np.random.RandomState(0).permutation(pages)).int().to(DEV)
    table = torch.full((3, room), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for step, new in enumerate([[40, 7, 130], [33, 100, 0], [1, 1, 1], [1, 1, 1], [2, 2, 2]]):
        n = sum(new)
        slots, cu_new, lens, cu_k, used = fa.fa_kv_assign(lens, i32(new), ps, table, free, n)
        free = free[int(used):].clone()
        k, v = randn_bf16(gen, heads, n, d), randn_bf16(gen, heads, n, d)
        fa.fa_kv_write_fp8(k.to(DEV), v.to(DEV), slots, kc, vc, ks, vs, k_bounds=kb)
        cache.write(f64(k), f64(v), slots.cpu().numpy())
        tab, length = table.cpu().numpy(), lens.cpu().tolist()
        if max(new) > 2:  # prompt chunks: the new rows attend over prefix and chunk
            total = sum(length)
            pk, pv = fa.fa_kv_read_fp8(kc, vc, ks, vs, table, cu_k, total)
            q = randn_bf16(gen, Hq, n, d)
            o, lse = fa.fa_fwd_varlen(q.to(DEV), pk, pv, cu_new, cu_k, max(new), max(length), True,
                                      scale)
            for b in range(3):
                lo, hi = sum(new[:b]), sum(new[:b + 1])
                if hi > lo:
                    ref = po.attend(f64(q)[None, :, lo:hi], cache, tab[b:b + 1], length[b:b + 1],
                                    scale)
                    assert np.abs(f64(o)[:, lo:hi] - ref[0][0]).max() <= 2e-2
                    assert np.abs(f64(lse)[:, lo:hi] - ref[1][0]).max() <= 1e-3
        else:
            Sq = new[0]
            q = randn_bf16(gen, 3, Hq, Sq, d)
            o, lse = fa.fa_decode_paged_fp8(q.to(DEV), kc, vc, ks, vs, table, lens, scale)
            check_attention(o, lse, po.attend(f64(q), cache, tab, length, scale), 400, d)
            sel, n_sel = fa.fa_select_blocks(q.to(DEV), kb, ks, table, lens, ps, 4)
            want = po.select(f64(q), cache.bounds, cache.scale[0], tab, length, ps, 4, 1, 1)
            assert np.array_equal(sel.cpu().numpy(), want[0])
            o, lse = fa.fa_decode_paged_fp8(q.to(DEV), kc, vc, ks, vs, table, lens, scale, sel=sel,
                                            n_sel=n_sel)
            check_attention(o, lse, po.attend(f64(q), cache, tab, length, scale, *want), 400, d)
    assert np.array_equal(kc.cpu().numpy(), cache.codes[0])
    assert np.array_equal(f64(ks), cache.scale[0])


def test_captured_step_replays_with_other_lengths():
    """One graph of a whole decode step; the replays see new lengths, tokens and pages."""
    heads, Hq, d, ps, room, B = 2, 4, 64, 16, 12, 3
    pages = B * room
    cache = make_cache(40, pages, heads, ps, d)
    dev = on_gpu(cache)
    free = torch.from_numpy(np.random.RandomState(1).permutation(pages)).int().to(DEV)
    base = np.full((B, room), -1, np.int32)
    table, seq, new = i32(base), i32([0] * B), i32([1] * B)
    k, v = (torch.empty(heads, B, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.empty(B, Hq, 1, d, dtype=torch.bfloat16, device=DEV)
    bufs = {}

    def step():
        slots, _, lens, _, used = fa.fa_kv_assign(seq, new, ps, table, free, B)
        fa.fa_kv_write_fp8(k, v, slots, *dev[:4], k_bounds=dev[4])
        sel, n_sel = fa.fa_select_blocks(q, dev[4], dev[2], table, lens, ps, 3)
        o, lse = fa.fa_decode_paged_fp8(q, *dev[:4], table, lens, 0.125, sel=sel, n_sel=n_sel)
        bufs.update(slots=slots, lens=lens, sel=sel, n_sel=n_sel, o=o, lse=lse)

    gen = torch.Generator().manual_seed(3)

    def load(lens):
        t = base.copy()
        at = pages - 1
        fr = free.cpu().numpy()
        for b, n in enumerate(lens):
            for i in range(po.pages_of(n, ps)):
                t[b, i] = fr[at]
                at -= 1
        table.copy_(i32(t))
        seq.copy_(i32(lens))
        kk, vv, qq = (randn_bf16(gen, heads, B, d), randn_bf16(gen, heads, B, d),
                      randn_bf16(gen, B, Hq, 1, d))
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        return t, kk, vv, qq

    def check(lens, t, kk, vv, qq):
        want = po.assign(lens, [1] * B, ps, t, free.cpu().numpy(), B)
        assert np.array_equal(bufs["slots"].cpu().numpy(), want[1])
        cache.write(f64(kk), f64(vv), want[1])
        ref_sel = po.select(f64(qq), cache.bounds, cache.scale[0], want[0], want[3], ps, 3, 1, 1)
        assert np.array_equal(bufs["sel"].cpu().numpy(), ref_sel[0])
        check_attention(bufs["o"], bufs["lse"],
                        po.attend(f64(qq), cache, want[0], want[3], 0.125, *ref_sel), 200, d)

    args = load([5, 0, 31])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # outside the capture
    torch.cuda.current_stream().wait_stream(stream)
    check([5, 0, 31], *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([16, 170, 3], [0, 0, 0], [100, 31, 15]):
        args = load(lens)
        graph.replay()
        torch.cuda.synchronize()
        check(lens, *args)


def test_back_to_back_steps_without_a_host_wait():
    """Lengths, tokens and lists change from call to call with nothing but the stream
    between them; every step's results equal those of the same steps taken one by one."""
    heads, Hq, d, ps, room, B = 2, 8, 64, 16, 40, 5
    pages = B * room
    gen = torch.Generator().manual_seed(70)
    start = [3, 200, 0, 77, 410]
    kv = [randn_bf16(gen, 2, heads, B, d).to(DEV) for _ in range(24)]
    qs = [randn_bf16(gen, B, Hq, 1, d).to(DEV) for _ in range(24)]

    def steps(wait):
        cache = make_cache(71, pages, heads, ps, d)
        dev = on_gpu(cache)
        table = i32(make_table(5, start, ps, pages, room=room))
        free = i32([p for p in range(pages) if p not in set(table.flatten().tolist())])
        lens, new, out, at = i32(start), i32([1] * B), [], 0
        filler = torch.zeros(1 << 22, device=DEV)
        for (k, v), q in zip(kv, qs):
            filler.add_(1.0)  # work for the next call's early launch to overlap with
            slots, _, lens, _, used = fa.fa_kv_assign(lens, new, ps, table, free, B)
            free = free[B:]   # one page for each request that might have taken one
            fa.fa_kv_write_fp8(k, v, slots, *dev[:4], k_bounds=dev[4])
            sel, n_sel = fa.fa_select_blocks(q, dev[4], dev[2], table, lens, ps, 6)
            if wait:
                torch.cuda.synchronize()
            a = fa.fa_decode_paged_fp8(q, *dev[:4], table, lens, 0.125)
            b = fa.fa_decode_paged_fp8(q, *dev[:4], table, lens, 0.125, sel=sel, n_sel=n_sel)
            out.append((lens, sel, *a, *b))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out

    for x, y in zip(steps(False), steps(True)):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_two_streams_at_once_with_workspaces_of_their_own():
    cache = make_cache(80, 300, 2, 16, 128)
    kc, vc, ks, vs, kb = on_gpu(cache)
    jobs = []
    for seed, lens, Sq in ((1, [2500, 1200], 1), (2, [900, 700, 1300], 4)):
        table = i32(make_table(seed, lens, 16, 300))
        q = randn_bf16(torch.Generator().manual_seed(seed), len(lens), 16, Sq, 128).to(DEV)
        ref = fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, i32(lens), 0.1)
        jobs.append((torch.cuda.Stream(), q, table, i32(lens), ref, []))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, table, lens, _, got in jobs:
            got.append(fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, lens, 0.1, stream=s))
    torch.cuda.synchronize()
    for *_, ref, got in jobs:
        for o, lse in got:
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_calls_on_a_side_stream_and_repeatability():
    lens = [3000, 10, 700]
    cache = make_cache(50, 250, 2, 16, 128)
    table = i32(make_table(1, lens, 16, 250))
    kc, vc, ks, vs, kb = on_gpu(cache)
    q = randn_bf16(torch.Generator().manual_seed(1), 3, 8, 1, 128).to(DEV)
    first = fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, i32(lens), 0.09)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):  # the same bits every time, on any stream
        o, lse = fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, i32(lens), 0.09, stream=s)
        s.synchronize()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_outputs_on_a_side_stream_are_not_memory_in_use():
    """Memory that the current stream freed, with its own writes still to come, must not
    become the output of a call on another stream."""
    lens = [300, 40]
    cache = make_cache(51, 30, 2, 16, 64)
    table = i32(make_table(1, lens, 16, 30))
    kc, vc, ks, vs, kb = on_gpu(cache)
    q, n = randn_bf16(torch.Generator().manual_seed(1), 2, 8, 1, 64).to(DEV), i32(lens)
    want = fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, n, 0.125)
    held = [torch.empty_like(w) for w in want]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    for t in held:
        t.fill_(7.0)
    del t, held
    got = fa.fa_decode_paged_fp8(q, kc, vc, ks, vs, table, n, 0.125, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sizes_past_32_bits_are_refused_by_the_calls():
    lens, table = i32([20, 3]), i32(np.zeros((2, 4)))
    with pytest.raises(ValueError, match="page_size"):
        fa.fa_kv_assign(lens, lens, (1 << 32) + 16, table, i32([0]), 4)
    with pytest.raises(ValueError, match="total_new"):
        fa.fa_kv_assign(lens, lens, 16, table, i32([0]), (1 << 32) + 4)
    kc, vc, ks, vs, kb = on_gpu(make_cache(1, 2, 1, 16, 64))
    with pytest.raises(ValueError, match="total_k"):
        fa.fa_kv_read_fp8(kc, vc, ks, vs, table, i32([0, 1, 2]), (1 << 32) + 2)
    q = torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(k_blocks=(1 << 32) + 2), dict(n_first=1 << 32), dict(n_last=1 << 32),
               dict(page_size=(1 << 32) + 16)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            fa.fa_select_blocks(q, kb, ks, table, lens, **{"page_size": 16, "k_blocks": 2, **kw})


def test_outputs_and_workspaces_are_all_that_is_written():
    guard = 4096

    def carve(shape, dtype):
        size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((2 * guard + size,), SENT, dtype=torch.uint8, device=DEV)
        bufs.append((buf, size))
        return buf[guard:guard + size].view(dtype).view(*shape)

    bufs = []
    B, Hq, heads, Sq, d, ps, lens = 3, 6, 2, 3, 64, 16, [70, 1, 250]
    pages, room = 24, 16
    cache = make_cache(60, pages, heads, ps, d)
    table = make_table(2, lens, ps, pages, room=room)
    kc, vc, ks, vs, kb = on_gpu(cache)
    dev = [carve(t.shape, t.dtype).copy_(t) for t in (kc, vc, ks, vs, kb)]
    tab = carve((B, room), torch.int32).copy_(i32(table))
    q = randn_bf16(torch.Generator().manual_seed(1), B, Hq, Sq, d).to(DEV)
    new = [3, 3, 3]
    free = i32([20, 21, 22, 23])
    slots, cu, out, cuk, used = fa.fa_kv_assign(
        i32(lens), i32(new), ps, tab, free, 11, slot_map=carve((11,), torch.int64),
        cu_new=carve((B + 1,), torch.int32), seqlens_out=carve((B,), torch.int32),
        cu_seqlens_k=carve((B + 1,), torch.int32), n_used=carve((1,), torch.int32))
    kv = randn_bf16(torch.Generator().manual_seed(2), 2, heads, 11, d).to(DEV)
    fa.fa_kv_write_fp8(kv[0], kv[1], slots, *dev[:4], k_bounds=dev[4])
    total = int(cuk[-1])
    fa.fa_kv_read_fp8(*dev[:4], tab, cuk, total, k=carve((heads, total, d), torch.bfloat16),
                      v=carve((heads, total, d), torch.bfloat16))
    sel, n_sel = fa.fa_select_blocks(
        q, dev[4], dev[2], tab, out, ps, 5, sel=carve((B, heads, 5), torch.int32),
        n_sel=carve((B, heads), torch.int32),
        workspace=carve((fa.fa_select_blocks_workspace_size(B, heads, room),), torch.uint8))
    for more in ({}, dict(sel=sel, n_sel=n_sel)):
        size = max(fa.fa_decode_paged_fp8_workspace_size(B, Hq, heads, Sq, d), 16)
        fa.fa_decode_paged_fp8(q, *dev[:4], tab, out, 0.125, o=carve(q.shape, torch.bfloat16),
                               lse=carve((B, Hq, Sq), torch.float32),
                               workspace=carve((size,), torch.uint8), **more)
    torch.cuda.synchronize()
    for buf, size in bufs:
        assert bool((buf[:guard] == SENT).all()) and bool((buf[guard + size:] == SENT).all())
