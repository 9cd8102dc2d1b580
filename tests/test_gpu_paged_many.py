"""GPU tests of the paged decode with thousands of requests, most of them short or empty (padded
batches): the results, and that the time grows no faster than the number of requests."""
import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import paged as po
from tests.paged import DEV, check_attention, f64, i32, make_cache, make_table, on_gpu, randn_bf16

pytestmark = pytest.mark.gpu


def _case(lens, Hq, heads, Sq, d, ps, seed, sel=None, n_sel=None):
    pages = sum(po.pages_of(n, ps) for n in lens) + 2
    cache = make_cache(seed, pages, heads, ps, d)
    table = make_table(seed + 1, lens, ps, pages)
    q = randn_bf16(torch.Generator().manual_seed(seed + 2), len(lens), Hq, Sq, d)
    ref = po.attend(f64(q), cache, table, lens, 0.125, sel, n_sel)
    more = {} if sel is None else dict(sel=i32(sel), n_sel=i32(n_sel))
    o = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], 9.0, device=DEV)
    fa.fa_decode_paged_fp8(q.to(DEV), *on_gpu(cache)[:4], i32(table), i32(lens), 0.125, o=o, lse=lse,
                           **more)
    torch.cuda.synchronize()
    check_attention(o, lse, ref, max(lens), d)


def _mostly_empty(B, places):
    lens = np.zeros(B, int)
    for b, n in places.items():
        lens[b] = n
    return lens.tolist()


@pytest.mark.parametrize("Hq,heads,Sq", [(8, 8, 1), (16, 8, 3), (24, 2, 1), (16, 2, 4), (20, 1, 2)])
@pytest.mark.parametrize("places", [{0: 900, 299: 2100}, {299: 5}, {7: 16, 8: 1, 150: 3000, 151: 17},
                                    {}, {0: 4000}])
def test_mostly_empty_batches(Hq, heads, Sq, places):
    _case(_mostly_empty(300, places), Hq, heads, Sq, 64, 16, seed=5)


@pytest.mark.parametrize("Hq,heads,Sq,d", [(4, 4, 1, 64), (36, 3, 1, 128), (8, 4, 9, 64)])
def test_thousands_of_short_requests(Hq, heads, Sq, d):
    rng = np.random.RandomState(Hq)
    lens = np.where(rng.rand(1100) < 0.4, 0, rng.randint(1, 45, 1100))
    lens[rng.randint(0, 1100, 3)] = 1500  # these lie in several CTAs' stretches
    _case(lens.tolist(), Hq, heads, Sq, d, 16, seed=6)


@pytest.mark.parametrize("Hq,Sq", [(4, 1), (12, 2), (36, 1)])
def test_chosen_blocks_of_many_requests(Hq, Sq):
    B, heads, ps, rng = 500, 2, 16, np.random.RandomState(3)
    lens = rng.randint(0, 200, B)
    sel, n_sel = np.full((B, heads, 9), -1), np.zeros((B, heads), int)
    for b in range(B):
        for h in range(heads):
            m = po.pages_of(int(lens[b]), ps)
            take = 0 if rng.rand() < 0.5 else min(m, rng.randint(0, 10))
            sel[b, h, :take] = np.sort(rng.permutation(m)[:take])
            n_sel[b, h] = take
    _case(lens.tolist(), Hq, heads, Sq, 64, ps, seed=7, sel=sel, n_sel=n_sel)


def _time(lens, Hq, heads, Sq):
    """Best time of a call in microseconds."""
    ps, d, B = 16, 64, len(lens)
    pages = max(sum(po.pages_of(n, ps) for n in lens), 1)
    cache = [torch.zeros(pages, heads, ps, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    cache += [torch.ones(pages, heads, device=DEV) for _ in range(2)]
    table, n = i32(make_table(1, lens, ps, pages)), i32(lens)
    q = torch.zeros(B, Hq, Sq, d, dtype=torch.bfloat16, device=DEV)
    out = dict(o=torch.empty_like(q), lse=torch.empty(B, Hq, Sq, device=DEV), workspace=torch.empty(
        max(fa.fa_decode_paged_fp8_workspace_size(B, Hq, heads, Sq, d), 16), dtype=torch.uint8,
        device=DEV))
    best = 1e9
    for _ in range(9):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda._sleep(200_000)  # the calls are queued before the first one begins
        a.record()
        for _ in range(4):
            fa.fa_decode_paged_fp8(q, *cache, table, n, 0.125, **out)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 4 * 1e3)
    return best


@pytest.mark.parametrize("Hq,Sq", [(8, 1), (32, 4)])
def test_empty_requests_cost_little(Hq, Sq):
    # 4096 requests of 8 KV heads of which two have keys: 10 ns for each (request, KV head) is
    # several times what reading their lengths and writing their rows takes
    few = _time([64, 64], Hq, 8, Sq)
    many = _time(_mostly_empty(4096, {0: 64, 4095: 64}), Hq, 8, Sq)
    assert many <= few + 328, f"{many:.0f} us against {few:.0f} us"


def test_time_grows_with_the_number_of_requests_no_faster():
    # eight times the requests: at most twice eight times the time
    a, b = (_time([16] * B, 32, 8, 8) for B in (500, 4000))
    assert b <= 16 * a, f"{b:.0f} us against {a:.0f} us"
