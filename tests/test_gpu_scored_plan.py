"""Mask plans: a plan of other sizes is refused, by the binding where it knows the plan's and on the device otherwise."""

import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from io_aware_exact_tcgen05_gb300 import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _plan(B, Sq, Sk, causal=True):
    return fa.fa_mask_plan(*fa.fa_row_bounds(B, Sq, Sk, causal), Sk)


@pytest.mark.parametrize("made,used", [
    # sizes whose plans have as many bytes: Sk within a tile, other rows and keys, another batch
    ((2, 300, 384), (2, 300, 300)), ((2, 300, 300), (2, 300, 384)), ((1, 46, 200), (1, 31, 500)),
    ((2, 21, 128), (1, 31, 500)), ((2, 6, 300), (1, 46, 200)),
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
