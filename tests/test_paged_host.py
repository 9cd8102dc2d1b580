"""Host-side checks of the paged-cache operators (no GPU): the oracle against
independent statements of its parts, and every refusal of the C ABI, which
comes before any device call."""
import ctypes

import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import build as fabuild
from oracle import paged as po

P = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def test_oracle_codes_match_torch_float8():
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(po.encode(x.double().numpy()), want.view(torch.uint8).numpy())
    codes = np.arange(256, dtype=np.uint8)
    back = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(po.decode_codes(codes), back, equal_nan=True)
    assert list(po.encode(np.array([np.inf, -np.inf, np.nan]))) == [0x7e, 0xfe, 0x7f]


@pytest.mark.parametrize("top", [448.0, 127.0])
def test_oracle_scale_is_the_smallest_power_that_fits(top):
    for amax in [1e-20, 0.3, 1.0, top, np.nextafter(top, 1e9), 2 * top, 1e20]:
        s = po.power_of_two_scale(amax, top)
        assert amax <= top * s and amax > top * s / 2
    assert po.power_of_two_scale(0.0, top) == 2.0 ** -100
    assert po.power_of_two_scale(1e-40, top) == 2.0 ** -100
    assert po.power_of_two_scale(3e38, top) <= 2.0 ** 119


def test_oracle_write_then_read_is_within_half_a_step():
    rng = np.random.RandomState(0)
    c = po.Cache(np.zeros((3, 2, 16, 64), np.uint8), np.zeros((3, 2, 16, 64), np.uint8),
                 np.zeros((3, 2)), np.zeros((3, 2)), np.zeros((3, 2, 2, 64)))
    k, v = rng.randn(2, 20, 64), rng.randn(2, 20, 64)
    slots = np.array([16 + i for i in range(16)] + [i for i in range(4)])
    c.write(k, v, slots)
    table = np.array([[1, 0]])
    for which, x in ((0, k), (1, v)):
        for h in range(2):
            got, absent = c.gather(which, table[0], h, np.arange(20))
            assert not absent.any()
            step = np.repeat(c.scale[which][[1, 0], h], [16, 4])[:, None] * 2.0 ** -9
            assert np.all(np.abs(got - x[h]) <= np.maximum(2.0 ** -4 * np.abs(x[h]), step / 2))
    for page, lo, n in ((1, 0, 16), (0, 16, 4)):
        y = po.decode_codes(c.codes[0][page, :, :n])
        assert np.all(4 * c.bounds[page, :, 0] >= y.max(axis=1))
        assert np.all(4 * c.bounds[page, :, 1] <= y.min(axis=1))


def test_oracle_attention_matches_torch():
    from tests.paged import make_cache, make_table
    lens, ps, d = [5, 40, 33], 16, 64
    c = make_cache(3, 8, 2, ps, d)
    table = make_table(1, lens, ps, 8)
    q = np.random.RandomState(2).randn(3, 4, 3, d)
    o, lse, *_ = po.attend(q, c, table, lens, 0.125)
    for b, n in enumerate(lens):
        for h in range(4):
            k = torch.from_numpy(c.gather(0, table[b], h // 2, np.arange(n))[0])
            v = torch.from_numpy(c.gather(1, table[b], h // 2, np.arange(n))[0])
            s = torch.from_numpy(q[b, h]) @ k.T * 0.125
            hide = torch.arange(n)[None] > torch.arange(3)[:, None] + n - 3
            s = s.masked_fill(hide, -np.inf)
            np.testing.assert_allclose(o[b, h], torch.softmax(s, 1) @ v, atol=1e-12)
            np.testing.assert_allclose(lse[b, h], torch.logsumexp(s, 1), atol=1e-12)


# ---------------------------------------------------------------- refusals --

def _assign(lib, **kw):
    a = dict(seq=0x1000, new=0x2000, B=2, ps=16, table=0x3000, room=4, free=0x4000, n_free=3,
             slots=0x5000, total=10, cu=0x6000, out=0x7000, cuk=0x8000, used=0x9000)
    a.update(kw)
    return lib.fa_kv_assign(P(a["seq"]), P(a["new"]), a["B"], a["ps"], P(a["table"]), a["room"],
                            P(a["free"]), a["n_free"], P(a["slots"]), a["total"], P(a["cu"]),
                            P(a["out"]), P(a["cuk"]), P(a["used"]), None)


@pytest.mark.parametrize("kw,word", [
    (dict(B=0), b"B=0"), (dict(room=0), b"max_blocks=0"), (dict(n_free=-1), b"n_free=-1"),
    (dict(total=-1), b"total_new=-1"), (dict(room=1 << 28), b"2^31"),
    (dict(seq=0), b"seqlens is NULL"), (dict(new=0x2002), b"newlens is not 4-byte"),
    (dict(table=0), b"block_table"), (dict(free=0), b"free_pages"), (dict(slots=0x5004), b"slot_map"),
    (dict(cu=0), b"cu_new"), (dict(out=0), b"seqlens_out"), (dict(cuk=0), b"cu_seqlens_k"),
    (dict(used=0), b"n_used"),
    (dict(out=0x1000), b"seqlens_out overlaps seqlens"),
    (dict(out=0x1004), b"seqlens_out overlaps seqlens"),
    (dict(slots=0x3ff8), b"slot_map overlaps free_pages"),
    (dict(table=0x1fe4), b"block_table overlaps newlens"),
])
def test_assign_refusals(lib, kw, word):
    assert _assign(lib, **kw) == fa.FA_ERR_INVALID_ARG
    assert word in lib.fa_last_error_detail()


def test_assign_refuses_page_sizes(lib):
    for ps in (0, 8, 24, 256, -16):
        assert _assign(lib, ps=ps) == fa.FA_ERR_UNSUPPORTED


def _write(lib, **kw):
    a = dict(k=16, v=16, kh=64, kt=64, vh=64, vt=64, slots=8, n=3, kc=16, vc=16, ks=4, vs=4, kb=16,
             pages=4, Hkv=2, ps=16, d=64)
    a.update(kw)
    return lib.fa_kv_write_fp8(P(a["k"]), P(a["v"]), a["kh"], a["kt"], a["vh"], a["vt"],
                               P(a["slots"]), a["n"], P(a["kc"]), P(a["vc"]), P(a["ks"]),
                               P(a["vs"]), P(a["kb"]), a["pages"], a["Hkv"], a["ps"], a["d"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(k=0), b"k is NULL"), (dict(v=8), b"v is not 16-byte"), (dict(kc=0), b"k_cache"),
    (dict(vc=24), b"v_cache"), (dict(ks=0), b"k_scale"), (dict(vs=2), b"v_scale"),
    (dict(kb=8), b"k_bounds"), (dict(slots=4), b"slot_map"), (dict(n=-1), b"n_tokens"),
    (dict(kh=4), b"strides"), (dict(vt=-64), b"strides"), (dict(pages=0), b"num_pages=0"),
    (dict(Hkv=0), b"Hkv=0"), (dict(Hkv=70000), b"65535"),
])
def test_write_refusals(lib, kw, word):
    assert _write(lib, **kw) == fa.FA_ERR_INVALID_ARG
    assert word in lib.fa_last_error_detail()


def test_write_refuses_shapes_and_accepts_no_tokens(lib):
    assert _write(lib, d=96) == fa.FA_ERR_UNSUPPORTED
    assert _write(lib, ps=48) == fa.FA_ERR_UNSUPPORTED
    assert _write(lib, n=0, k=0, v=0, slots=0) == fa.FA_OK


def _read(lib, **kw):
    a = dict(kc=16, vc=16, ks=4, vs=4, table=4, cu=4, k=16, v=16, nseq=2, room=3, pages=4, total=9,
             Hkv=2, ps=16, d=64)
    a.update(kw)
    return lib.fa_kv_read_fp8(P(a["kc"]), P(a["vc"]), P(a["ks"]), P(a["vs"]), P(a["table"]),
                              P(a["cu"]), P(a["k"]), P(a["v"]), a["nseq"], a["room"], a["pages"],
                              a["total"], a["Hkv"], a["ps"], a["d"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(kc=0), b"k_cache"), (dict(vc=0), b"v_cache"), (dict(ks=0), b"k_scale"),
    (dict(vs=0), b"v_scale"), (dict(table=0), b"block_table"), (dict(cu=2), b"cu_seqlens_k"),
    (dict(k=8), b"k is not"), (dict(v=0), b"v is NULL"), (dict(nseq=0), b"nseq=0"),
    (dict(room=0), b"max_blocks=0"), (dict(total=-1), b"total_k=-1"),
])
def test_read_refusals(lib, kw, word):
    assert _read(lib, **kw) == fa.FA_ERR_INVALID_ARG
    assert word in lib.fa_last_error_detail()
    assert _read(lib, total=0, k=0, v=0) == fa.FA_OK


def _select(lib, ws=256, nbytes=1 << 20, **kw):
    a = dict(q=16, kb=16, ks=4, table=4, lens=4, sel=4, n_sel=4, B=2, Hq=4, Hkv=2, Sq=1, pages=4,
             room=8, ps=16, d=64, k=4, first=1, last=1)
    a.update(kw)
    return lib.fa_select_blocks(P(a["q"]), P(a["kb"]), P(a["ks"]), P(a["table"]), P(a["lens"]),
                                P(a["sel"]), P(a["n_sel"]), a["B"], a["Hq"], a["Hkv"], a["Sq"],
                                a["pages"], a["room"], a["ps"], a["d"], a["k"], a["first"],
                                a["last"], P(ws), nbytes, None)


@pytest.mark.parametrize("kw,word", [
    (dict(q=8), b"q is not"), (dict(kb=0), b"k_bounds"), (dict(ks=0), b"k_scale"),
    (dict(table=0), b"block_table"), (dict(lens=0), b"seqlens_k"), (dict(sel=0), b"sel"),
    (dict(n_sel=0), b"n_sel"), (dict(k=0, first=0, last=0), b"k_blocks=0"),
    (dict(first=-1), b"n_first=-1"), (dict(last=4), b"n_last=4"), (dict(Hq=3), b"Hq (3)"),
    (dict(B=0), b"B=0"), (dict(Sq=0), b"Sq=0"), (dict(B=40000), b"65535"),
])
def test_select_refusals(lib, kw, word):
    assert _select(lib, **kw) == fa.FA_ERR_INVALID_ARG
    assert word in lib.fa_last_error_detail()


def test_select_workspace(lib):
    need = fa.fa_select_blocks_workspace_size(2, 2, 8)
    assert need >= 2 * 2 * 8 * 4
    assert _select(lib, nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert _select(lib, ws=0) == fa.FA_ERR_WORKSPACE
    assert _select(lib, ws=264) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_select_blocks_workspace_size(0, 2, 8) == 0


def _decode(lib, ws=256, nbytes=1 << 30, **kw):
    a = dict(q=16, kc=16, vc=16, ks=4, vs=4, table=4, lens=4, sel=0, n_sel=0, o=16, lse=0, B=2, Hq=4,
             Hkv=2, Sq=1, pages=4, room=8, max_sel=0, ps=16, d=64, scale=0.1)
    a.update(kw)
    return lib.fa_decode_paged_fp8(P(a["q"]), P(a["kc"]), P(a["vc"]), P(a["ks"]), P(a["vs"]),
                                   P(a["table"]), P(a["lens"]), P(a["sel"]), P(a["n_sel"]),
                                   P(a["o"]), P(a["lse"]), a["B"], a["Hq"], a["Hkv"], a["Sq"],
                                   a["pages"], a["room"], a["max_sel"], a["ps"], a["d"],
                                   F(a["scale"]), P(ws), nbytes, None)


@pytest.mark.parametrize("kw,word", [
    (dict(q=0), b"q is NULL"), (dict(kc=8), b"k_cache"), (dict(vc=0), b"v_cache"),
    (dict(ks=0), b"k_scale"), (dict(vs=0), b"v_scale"), (dict(table=0), b"block_table"),
    (dict(lens=2), b"seqlens_k"), (dict(o=0), b"o is NULL"), (dict(lse=8), b"lse is not"),
    (dict(sel=4), b"together"), (dict(n_sel=4), b"together"),
    (dict(sel=4, n_sel=4, max_sel=0), b"max_sel"), (dict(scale=-1.0), b"scale"),
    (dict(scale=float("inf")), b"scale"), (dict(Hq=5), b"Hq (5)"), (dict(Sq=-1), b"Sq=-1"),
    (dict(room=0), b"max_blocks=0"), (dict(room=1 << 28), b"2^31"), (dict(B=1 << 16), b"65535"),
])
def test_decode_refusals(lib, kw, word):
    assert _decode(lib, **kw) == fa.FA_ERR_INVALID_ARG
    assert word in lib.fa_last_error_detail()


def test_decode_refuses_shapes(lib):
    assert _decode(lib, d=80) == fa.FA_ERR_UNSUPPORTED
    assert _decode(lib, ps=8) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_decode_paged_fp8_workspace_size(1, 3, 2, 1, 64) == 0


def test_decode_rows_past_32_bits(lib):
    """65536 x 65537 rows are 65536 in 32 bits; 65536 x 32768 are negative there."""
    for Sq in (65537, 32768):
        assert fa.fa_decode_paged_fp8_workspace_size(1, 65536, 1, Sq, 64) == 0
        assert _decode(lib, B=1, Hq=65536, Hkv=1, Sq=Sq) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("x", [1 << 31, (1 << 32) + 16, -(1 << 31) - 1])
def test_sizes_past_32_bits_are_refused(x):
    with pytest.raises(ValueError, match="32 bits"):
        fa._int(x, "page_size")


def test_bindings_refuse_host_tensors(lib):
    z = torch.zeros
    with pytest.raises(TypeError):
        fa.fa_kv_assign(z(2, dtype=torch.int32), z(2, dtype=torch.int32), 16,
                        z(2, 3, dtype=torch.int32), z(4, dtype=torch.int32), 5)
    c = z(4, 2, 16, 64, dtype=torch.uint8)
    s = z(4, 2)
    with pytest.raises(TypeError):
        fa.fa_decode_paged_fp8(z(1, 2, 1, 64, dtype=torch.bfloat16), c, c, s, s,
                               z(1, 3, dtype=torch.int32), z(1, dtype=torch.int32), 0.1)
    with pytest.raises(TypeError):
        fa.fa_kv_write_fp8(z(2, 3, 64, dtype=torch.bfloat16), z(2, 3, 64, dtype=torch.bfloat16),
                           z(3, dtype=torch.int64), c, c, s, s)
