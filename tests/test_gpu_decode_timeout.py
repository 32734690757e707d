"""The bounded waits of fp2_decode, made to run out without faulting anything: a
copy that is never issued (debug_withhold_k_item) and a short limit
(debug_wait_limit_us).  Every wait ends, the error is reported, nothing is joined
from another call's records, and the next call on the workspace is right."""
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests.test_gpu_decode import Case

FORMS = [("bf16", 8, 1, 128, 1), ("fp8", 8, 1, 128, 2), ("bf16", 8, 2, 64, 4), ("bf16", 8, 1, 128, 4), ("fp8", 16, 2, 128, 4)]
LENS = [[9000], [60000, 50], [300] * 200]  # joined by item, by item with whole ones, by share


def withhold(p, item):
    p.params.debug_wait_limit_us = 20000 if item else 0
    p.params.debug_withhold_k_item = item


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,d,n", FORMS)
@pytest.mark.parametrize("lk,item", [(LENS[0], 1), (LENS[1], 1), (LENS[1], 2), (LENS[2], 1), (LENS[2], 2)])
def test_a_wait_that_runs_out(dtype, Hq, Hkv, d, n, lk, item):
    c = Case([n] * len(lk), lk, Hq, Hkv, d, 64, dtype, seed=50, pad=3)
    p = c.plan()
    p.out.fill_(5.0)
    p.lse.fill_(5.0)
    p.run()
    p.check()
    out, lse = p.out.clone(), p.lse.clone()
    withhold(p, item)
    p.out.fill_(3.0)
    p.lse.fill_(3.0)
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert e.value.status == fp2.FP2_ERR_TIMEOUT and 16 <= e.value.detail < 32
    rows = sum(c.lq)
    assert (p.out[rows:] == 3).all() and (p.lse[rows:] == 3).all()
    if item == 1:  # no CTA gets anywhere
        assert (p.out == 3).all() and (p.lse == 3).all()
    withhold(p, 0)
    p.out.fill_(5.0)
    p.lse.fill_(5.0)
    p.run()
    p.check()
    assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,d,n", FORMS)
def test_a_wait_that_runs_out_after_another_error(dtype, Hq, Hkv, d, n):
    """The error word holds an earlier error, the workspace an earlier call's records (of more
    sequences and rows): neither leads the join anywhere."""
    big = Case([n] * 3, [7000, 8000, 9000], Hq, Hkv, d, 64, dtype, seed=51)
    c = Case([n], [9000], Hq, Hkv, d, 64, dtype, seed=52, pad=3 * n)
    b = big.plan()
    p = c.plan(workspace=b.workspace)
    keep = int(big.table[1, 2])
    big.table[1, 2] = 10 ** 6
    b.run()
    big.table[1, 2] = keep
    withhold(p, 1)
    p.out.fill_(3.0)
    p.lse.fill_(3.0)
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 3)
    assert (p.out == 3).all() and (p.lse == 3).all()
    withhold(p, 0)
    p.run()
    c.check(p)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 4])
def test_an_unread_timeout_does_not_stop_the_next_call(n):
    c = Case([n], [9000], 8, 1, 128, 64, "bf16", seed=53)
    p = c.plan()
    withhold(p, 1)
    p.run()
    withhold(p, 0)
    p.out.fill_(3.0)
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert e.value.status == fp2.FP2_ERR_TIMEOUT
    c.check(p)
