"""Offsets and lengths whose sums or differences pass 32 bits are bad lengths to
the prefill, not short ones: recorded, and nothing of the output written."""
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2

pytestmark = pytest.mark.gpu
MAX, MIN = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("which,values", [
    ("cu", [MAX, MIN + 5, MIN + 6]),        # a difference that wraps to 6
    ("cu", [MAX - 2, MAX, MAX]),            # an end that wraps when added up
    ("cu", [MIN, MAX, MAX]),                # a difference that wraps to -1
    ("lens_k", [MIN, MIN + 7]),             # a prefix that wraps to a large one
    ("lens_k", [MAX, MAX]),
    ("cu_k", [MAX - 100, MAX - 50, MAX]),   # an end of keys that wraps
    ("cu_k", [MIN, MIN + 50, MIN + 90])])
def test_wrapping_offsets_are_bad_lengths(which, values, page, kernel):
    if which == "cu_k" and page:
        pytest.skip("paged keys have no offsets")
    lq, lk, Hq, Hkv, d = [200, 70], [328, 70], 8, 2, 128
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn((sum(lq), Hq, d), generator=g, device="cuda").bfloat16()
    rows = 512 if page else sum(lk)
    k, v = (torch.randn((rows, Hkv, d), generator=g, device="cuda").bfloat16() for _ in "kv")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t = {"cu": i32([0, 200, 270]), "lens_k": i32(lk), "cu_k": i32([0, 328, 398])}
    kw = dict(page_table=i32([[0, 1, 2, 3, 4, 5], [6, 7, 0, 0, 0, 0]]), page_size=page) if page else dict(cu_seqlens_k=t["cu_k"])
    if page:
        k, v = (x.view(-1, page, Hkv, d) for x in (k, v))
    pr = fp2.make_problem(q, k, v, t["cu"], Hq=Hq, Hkv=Hkv, d=d, block=128, dtype=fp2.FP2_BF16, max_seqlen_q=200, max_seqlen_k=328,
                          seqlens_k=t["lens_k"], **kw)
    pr.params.attn_kernel = kernel
    pr.prefill(float("inf"))
    pr.check()
    good = pr.out.clone()
    keep = t[which].clone()
    t[which].copy_(i32(values))
    pr.out.fill_(3.0)
    pr.prefill(float("inf"))
    st, det = fp2.get_status(pr.params)
    assert (st, det) == ((fp2.FP2_ERR_DEVICE_BOUNDS if which == "cu_k" else fp2.FP2_ERR_INVALID_ARG), 1)
    assert (pr.out == 3).all()
    t[which].copy_(keep)
    pr.prefill(float("inf"))
    pr.check()
    assert torch.equal(pr.out, good)
