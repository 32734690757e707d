"""fp2_decode where its arithmetic is at its edges: one key far above a long flat
tail, scales of 0, values that are not finite behind a token.  Inputs and bounds as in test_gpu_decode.py."""
import numpy as np
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests.test_gpu_decode import E4M3, Case

pytestmark = pytest.mark.gpu


def stored(c, x, name):
    """Rows [.., heads, d] in the case's type, by the heads' scales."""
    if c.dtype == "fp8":
        return (x / c.scales[name][:, None]).clamp(-448, 448).to(E4M3)
    return x.bfloat16()


def put(c, name, rows, x):
    """Values of some cache rows (before any block factor)."""
    flat = getattr(c, name).view(-1, c.Hkv, c.d)
    x = stored(c, x, name)
    if c.dtype == "fp8":
        flat.view(torch.uint8)[rows] = x.view(torch.uint8)
    else:
        flat[rows] = x


def sink(lq, lk, gap, dtype, Hq, Hkv, factors, noise, seed):
    """Key 0 of each sequence `gap` above all others, its value 0; the others' logits
    within a few `noise` of 0, their values near 1: the output is what the tail adds."""
    c = Case(lq, lk, Hq, Hkv, 128, 64, dtype, seed=seed, factors=factors)
    g = torch.Generator("cuda").manual_seed(900 + seed)
    u = torch.where(torch.rand((Hkv, 128), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    T = c.q.shape[0]
    q = 2 * u.repeat_interleave(Hq // Hkv, 0)[None] + 0.1 * torch.randn((T, Hq, 128), generator=g, device="cuda")
    c.q.view(torch.uint8).copy_(stored(c, q, "q").view(torch.uint8))
    for b, rows in enumerate(c.rows):
        shape = (len(rows), Hkv, 128)
        k, v = noise * torch.randn(shape, generator=g, device="cuda") / 2, 1 + 0.25 * torch.randn(shape, generator=g, device="cuda")
        k[0] = gap / (2 * 128 ** 0.5) * u / (c.fac["k"][b, 0][:, None] if factors else 1.0)
        v[0] = 0
        put(c, "k", rows, k)
        put(c, "v", rows, v)
    return c


@pytest.mark.parametrize("gap", [12.0, 15.0, 17.0])
@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("dtype,factors", [("bf16", False), ("fp8", False), ("fp8", True)])
def test_tail_under_a_sink(dtype, factors, n, gap):
    """A long tail is not lost beside one key of nearly all the weight, whatever rounds
    the weights, in one sequence over all CTAs ..."""
    c = sink([n], [40000], gap, dtype, 8, 1, factors, 0.02, seed=40)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("gap,noise", [(12.0, 0.0), (15.0, 0.0), (17.0, 0.5)])
@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("dtype,factors", [("bf16", False), ("fp8", False), ("fp8", True)])
def test_tails_under_sinks_of_whole_sequences(dtype, factors, n, gap, noise):
    """... and in a batch whose sequences lie in one CTA's share each, with the sink."""
    lk = (np.arange(40) * 7 + 2900).tolist()
    c = sink([n] * 40, lk, gap, dtype, 64, 8, factors, noise, seed=41)
    p = c.plan()
    p.run()
    # (a third of the sequences are compared: the 64-bit form walks them row by row)
    c.check(p, skip=[b for b in range(40) if b % 3])


@pytest.mark.parametrize("noise", [0.0, 0.02])
@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("dtype,factors", [("bf16", False), ("fp8", False), ("fp8", True)])
def test_tails_far_under_sinks(dtype, factors, n, noise):
    """18 below the largest logit fp16 weights keep their 11 bits where the largest stands alone."""
    lk = (np.arange(40) * 7 + 2900).tolist()
    for lens in (lk, [40000]):
        c = sink([n] * len(lens), lens, 18.0, dtype, 64, 8, factors, noise, seed=42)
        p = c.plan()
        p.run()
        c.check(p, skip=[b for b in range(40) if b % 3])


@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("lk", [[170, 40], [9000]])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_a_scale_of_zero_with_e4m3_output(n, lk, which):
    """A KV head (or query head) of zeros; without scales of its own the output is in the stored
    values' units: for v_scale 0 it is finite, what the other scales' outputs would be for 1."""
    c = Case([n] * len(lk), lk, 16, 2, 128, 16, "fp8", seed=43)
    p = c.plan(out_dtype=fp2.FP2_FP8_E4M3)
    p.run()
    c.check(p, out_scale=c.scales["v"].repeat_interleave(8))
    first = p.out.view(torch.uint8).clone()
    c.scales[which][0] = 0.0
    p.out.view(torch.uint8).fill_(0x7F)
    p.run()
    if which == "v":
        p.check()
        assert torch.equal(p.out.view(torch.uint8), first)
    else:
        c.check(p, out_scale=c.scales["v"].repeat_interleave(8))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [1, 4])
def test_an_output_scale_of_zero(dtype, n):
    """An output scale of 0 stores zeros (and the other heads as they are)."""
    c = Case([n, n], [170, 40], 8, 1, 128, 16, dtype, seed=44)
    sc = torch.linspace(0.002, 0.02, 8, device="cuda")
    p = c.plan(out_dtype=fp2.FP2_FP8_E4M3, out_scale=sc)
    p.run()
    c.check(p, out_scale=sc)
    first = p.out.view(torch.uint8).clone()
    sc[3] = 0.0
    p.run()
    p.check()
    first[:, 3] = 0
    assert torch.equal(p.out.view(torch.uint8), first)


@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("scale,factor", [(0.0, 1e-30), (0.0, 1.0), (1e-25, 1e-25)])
def test_logits_scales_whose_product_is_zero(n, scale, factor):
    """Every logit 0, whatever way the product of the scales becomes 0: the output is the mean of
    the values seen, and masked keys are not among them."""
    c = Case([n, n], [165, 37], 8, 1, 128, 16, "fp8", seed=45, factors=True)
    c.scales["k"][0] = scale
    c.fac["k"].fill_(factor)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,d,n,lk", [(8, 2, 128, 4, 130), (2, 2, 128, 16, 24), (8, 1, 128, 3, 1026), (4, 2, 128, 9, 9), (8, 1, 128, 5, 258),
                                           (8, 1, 64, 4, 130)])
def test_each_token_sees_its_own_keys_only(dtype, Hq, Hkv, d, n, lk):
    """Tokens t .. n - 1 overflowed, for every t: the rows below t keep their bits, the others show
    it, whether it is in their keys or their values."""
    if dtype == "fp8" and d == 64:
        pytest.skip("e4m3 is head dimension 128 only")
    c = Case([n, 1], [lk, 50], Hq, Hkv, d, 16, dtype, seed=46)
    p = c.plan()
    p.run()
    c.check(p)
    out, lse = p.out.clone(), p.lse.clone()
    for which in "kv":
        x = getattr(c, which).view(-1, Hkv, d)
        raw = x.view(torch.uint8) if dtype == "fp8" else x
        for bad in ([0x7F] if dtype == "fp8" else [float("nan"), float("inf")]):
            for t in range(1, n):
                keep = raw[c.rows[0][lk - n + t:]].clone()
                raw[c.rows[0][lk - n + t:]] = bad
                p.run()
                p.check()
                assert torch.equal(p.out[:t], out[:t]) and torch.equal(p.lse[:t], lse[:t]), (which, bad, t)
                assert not torch.isfinite(p.out[t:n].float()).any(), (which, bad, t)
                assert torch.equal(p.out[n], out[n]) and torch.equal(p.lse[n], lse[n])
                if which == "v":
                    assert torch.equal(p.lse[t:n], lse[t:n])
                else:
                    assert not torch.isfinite(p.lse[t:n]).any()
                raw[c.rows[0][lk - n + t:]] = keep
    p.run()
    p.check()
    assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("lens,status", [([100, 301, 300], fp2.FP2_ERR_INVALID_ARG), ([100, -1, 300], fp2.FP2_ERR_INVALID_ARG),
                                         ([100, 0, 300], fp2.FP2_ERR_INVALID_ARG)])
def test_bad_key_lengths_are_invalid_arguments(n, lens, status):
    """Above max_seqlen_k, or fewer keys than new tokens: detail 1, and the other sequences stand."""
    c = Case([n] * 3, [100, 200, 300], 8, 1, 128, 64, seed=47)
    p = c.plan()
    c.seqlens_k.copy_(torch.tensor(lens, dtype=torch.int32))
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (status, 1)
    c.check(p, skip=(1,))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("bf16", 64)])
@pytest.mark.parametrize("lk", [[1], [4], [5, 4], [127]])
@pytest.mark.parametrize("n", [1, 2, 4])
def test_a_cache_that_ends_with_its_keys(dtype, d, lk, n):
    """A contiguous cache of fewer rows than one copy takes: what lies behind it is no key."""
    if min(lk) < n:
        n = min(lk)
    c = Case([n] * len(lk), lk, 8, 1, d, 0, dtype, seed=48)
    rows = sum(lk)
    c.k, c.v = c.k[:rows], c.v[:rows]
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("spread", [0.5, 3.0])
@pytest.mark.parametrize("factor", [1e-3, 1e-5, 1e-7, 1e-12, "falling", "rising", "mixed"])
def test_blocks_of_small_values(factor, spread, n):
    """Value factors far below 1 (one scale for a head whose other sequences, or blocks, hold
    larger values): what they stand for keeps its precision."""
    lens = [3000, 40, 9000] if n == 1 else [3000, 40, 700]
    c = Case([n] * 3, lens, 8, 1, 128, 64, "fp8", seed=49, factors=True, spread=spread)
    f = c.fac["v"]
    steps = torch.linspace(0, 1, f.shape[1], device="cuda")[None, :, None]
    if factor == "falling":
        f *= 10 ** (-9 * steps)
    elif factor == "rising":
        f *= 10 ** (-9 * (1 - steps))
    elif factor == "mixed":
        f[:, ::3] *= 1e-4
    else:
        f *= factor
    p = c.plan()
    p.run()
    c.check(p)
