"""GPU tests of the bounds that the quantising write keeps: they enclose the page's codes."""
import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import paged as po
from tests.paged import DEV, f64, make_cache, on_gpu

pytestmark = pytest.mark.gpu


def _grow(cache, held, amax):
    """A token with largest magnitude amax[page, head] enters offset `held` of every page."""
    pages, heads, ps, d = cache.codes[0].shape
    gen = np.random.RandomState(7)
    k = gen.uniform(-0.1, 0.1, (heads, pages, d)) * amax.T[:, :, None]
    k[:, :, 5] = amax.T
    k = torch.from_numpy(k).to(torch.bfloat16).to(DEV)
    slots = torch.arange(pages, dtype=torch.int64, device=DEV) * ps + held
    kc, vc, ks, vs, kb = on_gpu(cache)
    fa.fa_kv_write_fp8(k, k.clone(), slots, kc, vc, ks, vs, k_bounds=kb)
    torch.cuda.synchronize()
    return f64(k), kc.cpu().numpy(), f64(ks), kb.cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("d", [64, 128])
def test_bounds_enclose_codes_whose_scale_is_no_power_of_two(d):
    """Growing from such a scale rounds held codes by a ratio that is no power of two, some of
    them away from zero: 448 * 0.99 becomes 448 again."""
    pages, heads, ps, held = 96, 3, 16, 9
    cache = make_cache(1, pages, heads, ps, d)
    rng = np.random.RandomState(2)
    # every magnitude occurs, next to the largest and alone
    cache.codes[0][:, :, :held] = rng.randint(0, 127, (pages, heads, held, d)) | (
        rng.randint(0, 2, (pages, heads, held, d)) << 7)
    only = rng.rand(pages, heads, 1, d) < 0.5
    cache.codes[0][:, :, 1:held] = np.where(only, 0, cache.codes[0][:, :, 1:held])
    was = np.float32(2.0 ** -6 / np.linspace(1.005, 1.995, pages * heads)).reshape(pages, heads)
    cache.scale[0] = was.astype(np.float64)
    cache.bounds = po.bounds_of_codes(cache.codes[0][:, :, :held])
    old = cache.bounds.copy()
    _, codes, scale, bounds = _grow(cache, held, np.full((pages, heads), 448 * 2.0 ** -6))
    assert np.all(scale == 2.0 ** -6)
    y = po.decode_codes(codes[:, :, :held + 1])
    assert np.all(4 * bounds[:, :, 0] >= y.max(axis=2)) and np.all(4 * bounds[:, :, 1] <= y.min(axis=2))
    # and are no looser than a code's rounding (half a step, 2^-4 of it) and one unit
    r = (was / 2.0 ** -6)[:, :, None]
    new = y[:, :, held]
    most = np.maximum(4 * old[:, :, 0] * r * np.where(old[:, :, 0] > 0, 1 + 2.0 ** -4, 1 - 2.0 ** -4), new)
    least = np.minimum(4 * old[:, :, 1] * r * np.where(old[:, :, 1] < 0, 1 + 2.0 ** -4, 1 - 2.0 ** -4), new)
    assert np.all(4 * bounds[:, :, 0] < most + 4) and np.all(4 * bounds[:, :, 1] > least - 4)


def test_bounds_of_scales_too_far_apart_for_their_ratio():
    """s_old / s below fp32's range: a bound that is not 0 stays 1 or -1, rounded outwards."""
    ps, d, pages = 16, 64, 4
    cache = po.Cache(np.zeros((pages, 1, ps, d), np.uint8), np.zeros((pages, 1, ps, d), np.uint8),
                     np.zeros((pages, 1)), np.zeros((pages, 1)), np.zeros((pages, 1, 2, d)))
    dev = on_gpu(cache)
    gen = torch.Generator().manual_seed(3)
    for off, n, mult, flat in ((0, 3, 1e-29, 0), (3, 2, 1e21, d // 2), (5, 1, 1e38, d - 8)):
        k = (torch.randn(1, pages * n, d, generator=gen) * mult).to(torch.bfloat16)
        k[:, :, :flat] = 0
        slots = [p * ps + off + i for p in range(pages) for i in range(n)]
        cache.write(f64(k), f64(k), slots)
        fa.fa_kv_write_fp8(k.to(DEV), k.to(DEV), torch.tensor(slots, device=DEV), *dev[:4],
                           k_bounds=dev[4])
        torch.cuda.synchronize()
        assert np.array_equal(f64(dev[2]), cache.scale[0])
        assert np.array_equal(dev[4].cpu().numpy().astype(np.int64), cache.bounds)
