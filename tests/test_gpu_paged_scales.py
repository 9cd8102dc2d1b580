"""GPU tests of the paged decode where a KV head's pages have V scales far apart: what a
row gets from a page depends on that row's own weights there, not on how loud a page is that
has no weight or that the row does not see."""
import math

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import paged as po
from tests.paged import f64, i32, make_cache, make_table, on_gpu, randn_bf16, DEV

pytestmark = pytest.mark.gpu

ROWS = [(4, 2, 1), (2, 1, 3), (24, 2, 1), (6, 2, 4), (40, 1, 1), (9, 1, 4)]  # Hq, Hkv, Sq


def _terms(q, cache, table, lens, scale):
    """Per row: the largest weight * V scale of its visible keys (softmax weights)."""
    B, Hq, Sq, _ = q.shape
    heads, ps = cache.codes[0].shape[1:3]
    peak = np.zeros((B, Hq, Sq))
    for b, n in enumerate(lens):
        pos = np.arange(n)
        for h in range(heads):
            k, absent = cache.gather(0, table[b], h, pos)
            vs = cache.scale[1][np.where(absent, 0, table[b][pos // ps]), h]
            for g in range(h * (Hq // heads), (h + 1) * (Hq // heads)):
                for i in range(Sq):
                    see = ~absent & (pos <= i + n - Sq)
                    if see.any():
                        x = k[see] @ q[b, g, i] * scale
                        w = np.exp(x - x.max())
                        peak[b, g, i] = (w / w.sum() * vs[see]).max()
    return peak


def _check(cache, table, lens, q, scale):
    """Element-wise bound of O against the 64-bit values.

    A score is off by at most (d + 4) * 2^-24 of sum |q k|, and so is a weight by twice that,
    relatively.  The exponent of a stored weight is score + log2(V scale) - reference: four
    roundings to fp32 (half a unit each) of numbers no larger than |score| / ln 2 + 9 + the
    largest |log2 V scale|, and log2 itself two units (2^-22 near 1).  The stored weight is
    rounded to f16 (2^-11) or, far below the row's largest weight * V scale, by at most 2^-34
    of that, times codes of up to 448.  Exponentials and that log2 are off by 2^-20 together,
    sums run in fp32 (n * 2^-24), O is rounded to bf16 (2^-8)."""
    d, n = q.shape[-1], max(lens)
    ref, ref_lse, spread, size, _ = po.attend(f64(q), cache, table, lens, scale)
    peak = _terms(f64(q), cache, table, lens, scale)
    dev = on_gpu(cache)
    o, lse = fa.fa_decode_paged_fp8(q.to(DEV), *dev[:4], i32(table), i32(lens), scale)
    torch.cuda.synchronize()
    o, lse = f64(o), f64(lse)
    eps = 2.0 ** -24
    logs = np.abs(np.log2(cache.scale[1], where=cache.scale[1] > 0,
                          out=np.zeros_like(cache.scale[1]))).max()
    rel = (2 * (d + 4) * eps * size + 8 * eps * (1.45 * size + 9 + logs) + 2.0 ** -11 + 2.0 ** -20
           + n * eps)
    tol = 2.0 ** -8 * np.abs(ref) + rel[..., None] * spread * (1 + 2.0 ** -8) + (
        n * 448 * 2.0 ** -34 * peak[..., None])
    worst = (np.abs(o - ref) / np.maximum(tol, 1e-300)).max()
    assert worst <= 1.0, f"O is off by {worst:.2f} of its bound"
    seen = ref_lse > -np.inf
    assert np.array_equal(lse > -np.inf, seen)
    lse, ref_lse = np.where(seen, lse, 0.0), np.where(seen, ref_lse, 0.0)
    tol_l = (d + 4) * eps * size + (n + 8) * eps + 2.0 ** -21 + 4 * eps * np.abs(ref_lse)
    assert (np.abs(lse - ref_lse) <= tol_l).all(), "LSE"


def _steered(seed, pages, heads, ps, d, lens, offsets):
    """A cache whose page of block i has every key at about offsets(b, i) * 64 / 8 in the score
    of a query whose channel 0 is 64; offsets in [-3.5, 3.5]."""
    cache = make_cache(seed, pages, heads, ps, d)
    table = make_table(seed + 1, lens, ps, pages)
    for b, n in enumerate(lens):
        for i in range(po.pages_of(n, ps)):
            page = table[b, i]
            s = cache.scale[0][page][:, None]
            cache.codes[0][page, :, :, 0] = po.encode(offsets(b, i) / s)
    return cache, table


def _query(seed, B, Hq, Sq, d):
    q = randn_bf16(torch.Generator().manual_seed(seed), B, Hq, Sq, d)
    q[..., 0] = 64.0
    return q


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", ROWS)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_loud_page_without_weight_takes_nothing_from_the_others(d, Hq, heads, Sq, where):
    ps, lens = 16, [500, 90]
    at = [{"first": 0, "middle": po.pages_of(n, ps) // 2, "last": po.pages_of(n, ps) - 1}[where]
          for n in lens]
    cache, table = _steered(100, 40, heads, ps, d, lens,
                            lambda b, i: -3.0 if i == at[b] else 3.0)
    for b, i in enumerate(at):  # weight about 2^-69, 2^40 louder
        cache.scale[1][table[b, i]] *= 2.0 ** 40
    _check(cache, table, lens, _query(1, 2, Hq, Sq, d), 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", [(2, 1, 3), (1, 1, 6), (6, 2, 4), (9, 1, 4), (20, 1, 2)])
def test_a_loud_page_that_a_row_does_not_see_takes_nothing_from_it(d, Hq, heads, Sq):
    # the newest key begins a page of its own: all rows but the last do not see it
    ps, lens = 16, [16 * 20 + 1, 17]
    cache, table = _steered(110, 24, heads, ps, d, lens, lambda b, i: 0.0)
    for b, n in enumerate(lens):
        cache.scale[1][table[b, (n - 1) // ps]] *= 2.0 ** 45
    _check(cache, table, lens, _query(2, 2, Hq, Sq, d), 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", ROWS)
def test_light_loud_pages_and_heavy_quiet_ones_count_alike(d, Hq, heads, Sq):
    # weight * V scale is about the same for every page: from 2^-40 with all the weight to 2^40
    ps, lens = 16, [700, 130]
    off = lambda b, i: (i * 7 % 11 - 5) * 0.5  # noqa: E731
    cache, table = _steered(120, 60, heads, ps, d, lens, off)
    for b, n in enumerate(lens):
        for i in range(po.pages_of(n, ps)):
            cache.scale[1][table[b, i]] *= 2.0 ** round(-off(b, i) * 8 / math.log(2))
    _check(cache, table, lens, _query(3, 2, Hq, Sq, d), 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,heads,Sq", ROWS)
def test_scales_over_their_whole_range(d, Hq, heads, Sq):
    # 2^-100 to 2^119 at random, some no powers of two, some 0 (pages that were never written)
    ps, lens = 16, [5000, 333, 16, 1]
    rng = np.random.RandomState(5)
    cache, table = _steered(130, 360, heads, ps, d, lens, lambda b, i: rng.uniform(-3.4, 3.4))
    s = 2.0 ** rng.randint(-100, 112, cache.scale[1].shape)
    s = np.where(rng.rand(*s.shape) < 0.3, s * rng.uniform(1, 2, s.shape), s)
    cache.scale[1] = np.where(rng.rand(*s.shape) < 0.1, 0.0, np.float32(s).astype(np.float64))
    _check(cache, table, lens, _query(4, 4, Hq, Sq, d), 0.125)


@pytest.mark.parametrize("Hq,heads,Sq", ROWS)
def test_values_of_zero_scale_give_zero(Hq, heads, Sq):
    ps, d, lens = 16, 64, [300, 5]
    cache, table = _steered(140, 22, heads, ps, d, lens, lambda b, i: 0.0)
    cache.scale[1] = np.zeros_like(cache.scale[1])
    _check(cache, table, lens, _query(5, 2, Hq, Sq, d), 0.125)
