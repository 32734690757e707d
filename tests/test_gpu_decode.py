"""fp2_decode against a plain 64-bit attention: types, head layouts, page sizes,
lengths from one key to long ones, ragged batches, several new tokens, masked
keys that hold NaN, padded rows, errors, graphs, streams, shared workspaces."""
import numpy as np
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests import serve_ref as R

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


class Case:
    """Seeded inputs of one call on the GPU, stale rows of the cache full of NaN."""

    def __init__(self, lq, lk, Hq=8, Hkv=2, d=128, page=64, dtype="bf16", seed=0, factors=False, block=128, pad=0, spread=2.0,
                 stale=float("nan")):
        self.lq, self.lk, self.Hq, self.Hkv, self.d, self.page, self.dtype, self.block = lq, lk, Hq, Hkv, d, page, dtype, block
        rs = np.random.RandomState(1000 + seed)
        g = torch.Generator("cuda").manual_seed(seed)
        dev = "cuda"
        kind = E4M3 if dtype == "fp8" else torch.bfloat16
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32, device=dev)
        self.seqlens_k = torch.tensor(lk, dtype=torch.int32, device=dev)
        T = sum(lq) + pad
        self.scales = {n: 0.01 * (1 + torch.rand(h, generator=g, device=dev)) if dtype == "fp8" else torch.ones(h, device=dev)
                       for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}

        def values(shape, name, size):
            x = size * torch.randn(shape, generator=g, device=dev)
            return (x / self.scales[name][None, :, None]).clamp(-448, 448).to(kind) if dtype == "fp8" else x.to(kind)
        self.q = values((T, Hq, d), "q", spread)
        if page:
            need = [R.pages(n, page) for n in lk]
            perm = rs.permutation(sum(need) + 3)
            table = np.full((len(lk), max(1, max(need))), -1, np.int32)
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = perm[at:at + n]
                at += n
            self.table = torch.tensor(table, device=dev)
            rows, self.cu_k = len(perm) * page, None
            self.rows = [torch.tensor((table[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page), device=dev)
                         for b, n in enumerate(lk)]
        else:
            self.table, rows = None, sum(lk) + 5
            cu = np.concatenate([[0], np.cumsum(lk)])
            self.cu_k = torch.tensor(cu, dtype=torch.int32, device=dev)
            self.rows = [torch.arange(cu[b], cu[b + 1], device=dev) for b in range(len(lk))]
        self.k, self.v = (torch.full((rows, Hkv, d), stale, device=dev).to(kind) for _ in "kv")
        for x, n in ((self.k, "k"), (self.v, "v")):
            for r in self.rows:
                if len(r):
                    x.view(torch.uint8 if dtype == "fp8" else kind)[r] = values((len(r), Hkv, d), n, 1.0).view(torch.uint8 if dtype == "fp8" else kind)
        if page:
            self.k, self.v = (x.view(-1, page, Hkv, d) for x in (self.k, self.v))
        self.fac = {n: 1 - 0.75 * torch.rand((len(lk), R.pages(max(lk), block), Hkv), generator=g, device=dev) if factors else None for n in "kv"}

    def plan(self, **kw):
        fp8 = self.dtype == "fp8"
        args = dict(Hq=self.Hq, Hkv=self.Hkv, d=self.d, block=self.block, dtype=fp2.FP2_FP8_E4M3 if fp8 else fp2.FP2_BF16,
                    max_seqlen_q=max(1, max(self.lq)), max_seqlen_k=max(self.lk), seqlens_k=self.seqlens_k, cu_seqlens_k=self.cu_k,
                    page_table=self.table, page_size=self.page, k_block_factor=self.fac["k"], v_block_factor=self.fac["v"], with_lse=True)
        if fp8:
            args.update(q_scale=self.scales["q"], k_scale=self.scales["k"], v_scale=self.scales["v"])
        args.update(kw)
        return fp2.make_decode(self.q, self.k, self.v, self.cu, **args)

    def seq(self, b):
        """q, K, V of sequence b in float64, dequantised."""
        def rows(x, r):
            x = x.view(-1, x.shape[-2], x.shape[-1])
            return (x.view(torch.uint8)[r].view(E4M3) if self.dtype == "fp8" else x[r]).double()
        a = int(self.cu[b])
        q = self.q[a:a + self.lq[b]].double() * self.scales["q"].double()[:, None]
        K, V = rows(self.k, self.rows[b]), rows(self.v, self.rows[b])
        if self.dtype == "fp8":
            K, V = K * self.scales["k"].double()[:, None], V * self.scales["v"].double()[:, None]
        if self.fac["k"] is not None:
            n = len(self.rows[b])
            K, V = (x * self.fac[f][b].double().repeat_interleave(self.block, 0)[:n, :, None] for x, f in ((K, "k"), (V, "v")))
        return q, K, V

    def check(self, plan, skip=(), out_scale=None):
        plan.check()
        out_type = plan.out.dtype
        for b in range(len(self.lq)):
            if b in skip or not self.lq[b]:
                continue
            q, K, V = self.seq(b)
            ref, lse, absv, dot = R.decode(q, K, V, self.Hq // self.Hkv)
            unit = out_scale.double() if out_scale is not None else None
            tol, tol_lse = R.decode_bounds(ref, absv, dot, self.lk[b], self.d, self.dtype, out_type, unit)
            if unit is not None:
                ref = (ref / unit[:, None]).clamp(-448, 448)
            a = int(self.cu[b])
            got, got_lse = plan.out[a:a + self.lq[b]].double(), plan.lse[a:a + self.lq[b]].double()
            assert torch.isfinite(got).all() and torch.isfinite(got_lse).all(), b
            # (a bound of 0, where every value is 0, asks for the value itself)
            off, off_lse = (got - ref).abs(), (got_lse - lse).abs()
            assert (off <= tol).all(), (b, float((off / tol).nan_to_num(0).max()), float(off.max()))
            assert (off_lse <= tol_lse).all(), (b, float((off_lse / tol_lse).max()))


SHAPES = [(4, 1, 64), (2, 2, 64), (16, 2, 64), (8, 2, 128), (4, 4, 128), (4, 2, 128), (8, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("page", [0, 16, 64, 256])
def test_single_tokens_ragged(Hq, Hkv, d, page):
    lk = [1, 2, 15, 16, 17, 63, 64, 65, 129, 1000]
    c = Case([1] * len(lk), lk, Hq, Hkv, d, page, seed=1)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2), (8, 4), (16, 2)])
@pytest.mark.parametrize("page,factors", [(0, False), (16, True), (64, False), (128, True)])
def test_e4m3(Hq, Hkv, page, factors):
    lk = [1, 31, 32, 33, 127, 128, 500, 1]
    c = Case([1] * len(lk), lk, Hq, Hkv, 128, page, "fp8", seed=2, factors=factors)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 8), (8, 1), (4, 2)])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_several_tokens(dtype, Hq, Hkv, page):
    lq = [1, 16, 0, 5, 2, 3, 9, 7, 4]
    lk = [40, 16, 77, 5, 1200, 130, 21, 64, 259]
    c = Case(lq, lk, Hq, Hkv, 128, page, dtype, seed=3)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype,Hq,Hkv,lk", [("bf16", 4, 1, [20000]), ("fp8", 8, 1, [20011, 3, 9000]), ("bf16", 8, 8, [6000, 6001]),
                                             ("bf16", 2, 2, [33000, 1, 1, 15])])
def test_long_keys_are_split_and_joined(dtype, Hq, Hkv, lk):
    c = Case([1] * len(lk), lk, Hq, Hkv, 128, 64, dtype, seed=4)
    p = c.plan()
    p.run()
    c.check(p)
    first = p.out.clone(), p.lse.clone()
    p.workspace[256:].fill_(0xFF)  # what the workspace holds between calls does not matter
    p.run()
    p.check()
    assert torch.equal(first[0], p.out) and torch.equal(first[1], p.lse)


def test_many_sequences():
    rs = np.random.RandomState(5)
    lk = rs.randint(1, 90, 700).tolist()
    lq = [min(k, int(n)) for k, n in zip(lk, rs.randint(0, 3, 700))]
    c = Case(lq, lk, 4, 2, 128, 16, seed=5)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_sharp_and_flat_rows(dtype):
    """Logits far apart (one key takes all) and all equal (out is the mean)."""
    c = Case([1, 1], [700, 4097], 8, 2, 128, 64, dtype, seed=6, spread=30.0)
    p = c.plan()
    p.run()
    c.check(p)
    c.q.zero_()
    p.run()
    c.check(p)
    assert torch.allclose(p.lse[1], torch.full_like(p.lse[1], float(np.log(4097))), atol=1e-5)


@pytest.mark.parametrize("scale_given", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_e4m3_output(dtype, scale_given):
    if dtype == "bf16" and not scale_given:
        pytest.skip("bf16 inputs need a scale")
    c = Case([1, 2], [300, 2000], 8, 2, 128, 64, dtype, seed=7)
    sc = torch.linspace(0.002, 0.02, 8, device="cuda") if scale_given else None
    p = c.plan(out_dtype=fp2.FP2_FP8_E4M3, out_scale=sc)
    p.run()
    c.check(p, out_scale=sc if scale_given else c.scales["v"].repeat_interleave(4))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,n,lk", [(8, 2, 4, 130), (2, 2, 16, 24), (8, 1, 3, 1026), (4, 2, 9, 9)])
def test_masked_keys_hold_nan(dtype, Hq, Hkv, n, lk):
    """A drafted token that overflowed leaves the tokens before it alone, whether
    its key or its value is not finite; the rows that see it become NaN."""
    bads = [float("nan")] if dtype == "fp8" else [float("nan"), float("inf")]
    for bad in bads:
        for which in "kv":
            c = Case([n, 1], [lk, 50], Hq, Hkv, 128, 16, dtype, seed=8)
            clean = c.plan()
            clean.run()
            c.check(clean)
            ref, ref_lse = clean.out.clone(), clean.lse.clone()
            x = getattr(c, which).view(-1, Hkv, 128)
            for t in range(1, n):  # poison the last n - t tokens: rows below t stay
                raw = x.view(torch.uint8) if dtype == "fp8" else x
                raw[c.rows[0][lk - n + t]] = 0x7F if dtype == "fp8" else bad
            p = c.plan()
            p.run()
            p.check()
            assert torch.equal(p.out[0], ref[0]) and torch.equal(p.lse[0], ref_lse[0])
            assert torch.equal(p.out[n], ref[n])
            if which == "v":
                assert not torch.isfinite(p.out[1:n].float()).any()


def test_rows_behind_the_last_sequence_stay():
    c = Case([1, 0, 2], [100, 40, 60], pad=3, seed=9)
    p = c.plan()
    p.out.fill_(7.0)
    p.lse.fill_(8.0)
    p.run()
    c.check(p)
    assert (p.out[3:] == 7).all() and (p.lse[3:] == 8).all()


def test_no_lse_and_no_tokens():
    c = Case([1], [100], seed=10)
    p = c.plan(with_lse=False)
    p.run()
    assert p.lse is None
    q = c.plan()
    q.run()
    q.check()
    assert torch.equal(p.out, q.out)
    c = Case([0, 0], [100, 3], seed=10, pad=2)
    p = c.plan()
    p.out.fill_(3.0)
    p.run()
    p.check()
    assert (p.out == 3).all()


def test_device_errors_are_recorded_and_leave_the_rest():
    c = Case([1, 1, 1], [100, 200, 300], seed=11)
    p = c.plan()
    c.seqlens_k[1] = 301  # above max_seqlen_k
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert e.value.status == fp2.FP2_ERR_DEVICE_BOUNDS or e.value.status == fp2.FP2_ERR_INVALID_ARG
    c.seqlens_k[1] = 200
    p.run()
    c.check(p)
    keep = int(c.table[1, 2])
    for bad in (-1, 10 ** 6):
        c.table[1, 2] = bad
        p.run()
        with pytest.raises(fp2.Fp2Error) as e:
            p.check()
        assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 3)
        c.check(p, skip=(1,))
    c.table[1, 2] = keep
    p.run()
    c.check(p)


def test_bad_scale_factor_is_recorded():
    c = Case([1, 1], [300, 200], 8, 2, 128, 64, "fp8", seed=12, factors=True)
    p = c.plan()
    c.fac["v"][0, 1, 1] = 1.5
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_INVALID_ARG, 5)


def test_captured_graph_follows_the_lengths():
    """Replays see the lengths, table and rows that the buffers hold then, and
    another stream than the capture's may have filled them."""
    c = Case([1, 1, 1], [70, 900, 3000], seed=13, page=64)
    p = c.plan()
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for lens in ([70, 900, 3000], [1, 64, 65], [70, 1, 2999]):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.seqlens_k.copy_(torch.tensor(lens, dtype=torch.int32))
            p.out.zero_()
        torch.cuda.current_stream().wait_stream(side)
        g.replay()
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.lk, d.rows = lens, [r[:n] for r, n in zip(c.rows, lens)]
        d.check(p)


def test_two_graphs_share_a_workspace():
    a = Case([1], [5000], 8, 2, 128, 64, seed=14)
    b = Case([2, 1], [900, 7000], 8, 1, 128, 64, seed=15)
    pa = a.plan()
    pb = b.plan(workspace=pa.workspace)
    graphs = []
    for p in (pa, pb):
        p.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    for _ in range(3):
        for p, g in zip((pa, pb), graphs):
            p.out.zero_()
            g.replay()
    a.check(pa)
    b.check(pb)


def test_other_stream():
    c = Case([1, 1], [500, 4000], seed=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p = c.plan()
        p.run()
    s.synchronize()
    c.check(p)
    fixed = c.plan(stream=s.cuda_stream)
    torch.cuda.synchronize()
    fixed.run()
    s.synchronize()
    assert torch.equal(fixed.out, p.out)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 values (and 2^32 bytes): pages at its far end."""
    Hq, Hkv, d, page = 8, 8, 128, 64
    npages = 2 ** 31 // (page * Hkv * d) + 100
    c = Case([1, 1], [200, 300], Hq, Hkv, d, page, seed=17)
    k, v = (torch.empty((npages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = c.table.clone()
    ids = c.table[c.table >= 0].long()
    for x, y in ((k, c.k), (v, c.v)):
        x[npages - 50 + ids] = y[ids]
    table[table >= 0] += npages - 50
    p = c.plan()
    p.run()
    c.check(p)
    far = fp2.make_decode(c.q, k, v, c.cu, Hq=Hq, Hkv=Hkv, d=d, dtype=fp2.FP2_BF16, max_seqlen_q=1, max_seqlen_k=300,
                          seqlens_k=c.seqlens_k, page_table=table, page_size=page, with_lse=True)
    far.run()
    far.check()
    assert torch.equal(far.out, p.out) and torch.equal(far.lse, p.lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_equals_the_prefill_with_every_block_kept(dtype):
    """The framework's own attention on the same cache, at tau = inf: both are
    within their roundings of the same function (fp8: the prefill rounds its
    weights to e4m3, 2^-4 of each, which is its own stated tolerance)."""
    c = Case([1, 3], [400, 700], 8, 2, 128, 64, dtype, seed=18, stale=0.0)
    p = c.plan()
    p.run()
    c.check(p)
    pr = fp2.make_problem(c.q, c.k, c.v, c.cu, Hq=8, Hkv=2, d=128, block=128, dtype=p.dtype, max_seqlen_q=3, max_seqlen_k=700,
                          seqlens_k=c.seqlens_k, page_table=c.table, page_size=64,
                          **({n + "_scale": c.scales[n] for n in "qkv"} if dtype == "fp8" else {}))
    pr.prefill(float("inf"))
    pr.check()
    a, b = p.out.double(), pr.out.double()
    assert float((a - b).norm() / b.norm()) <= (5e-2 if dtype == "fp8" else 5e-3) + 2.0 ** -8


@pytest.mark.parametrize("dtype,Hq,Hkv,n,page,factors", [("bf16", 64, 8, 4, 64, False), ("fp8", 64, 8, 4, 64, True), ("fp8", 8, 1, 16, 16, False),
                                                        ("bf16", 4, 1, 9, 256, False), ("fp8", 16, 2, 3, 128, True), ("bf16", 3, 3, 16, 0, False)])
def test_drafts_over_long_keys(dtype, Hq, Hkv, n, page, factors):
    """Several tokens over keys that many CTAs share: partial results of whole
    tiles, tiles that end inside a page, new keys on both sides of a tile's edge."""
    lk = [9000, 128 + n // 2, 256, 1023, n, 4097]
    c = Case([n, n, n, 1, n, 2], lk, Hq, Hkv, 128, page, dtype, seed=20, factors=factors)
    p = c.plan()
    p.run()
    c.check(p)
    first = p.out.clone(), p.lse.clone()
    p.workspace[256:].fill_(0xFF)
    p.run()
    p.check()
    assert torch.equal(first[0], p.out) and torch.equal(first[1], p.lse)


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 4), (8, 1, 16), (2, 2, 16), (4, 1, 2)])
def test_drafts_at_head_dimension_64(Hq, Hkv, n):
    c = Case([n, 1, n], [3000, 40, n + 7], Hq, Hkv, 64, 32, "bf16", seed=21)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 1), (8, 1, 2), (16, 2, 5)])
def test_rising_logits(dtype, Hq, Hkv, n):
    """Logits that grow along the keys by far more than a weight may: the running
    reference moves again and again, and the early keys' weights vanish."""
    c = Case([n], [3000], Hq, Hkv, 128, 64, dtype, seed=22, spread=4.0)
    flat = c.k.view(-1, Hkv, 128)
    ramp = torch.linspace(0.02, 6.0, 3000, device="cuda")[:, None, None]
    q = c.q.double().mean(0).sign().view(Hkv, Hq // Hkv, 128)[:, 0]  # keys along one row's signs
    rows = (q[None] * ramp).float()
    if dtype == "fp8":
        raw = (rows / c.scales["k"][None, :, None]).clamp(-448, 448).to(E4M3)
        flat.view(torch.uint8)[c.rows[0]] = raw.view(torch.uint8)
    else:
        flat[c.rows[0]] = rows.bfloat16()
    p = c.plan()
    p.run()
    c.check(p)


def test_many_drafting_sequences():
    rs = np.random.RandomState(23)
    lk = rs.randint(20, 400, 300).tolist()
    lq = rs.randint(0, 6, 300).tolist()
    lq[7] = 6
    c = Case(lq, lk, 8, 1, 128, 16, "fp8", seed=23)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_drafts_in_a_captured_graph(dtype):
    """Replays with other numbers of drafted tokens than at the capture."""
    c = Case([4, 4, 4], [2000, 300, 700], 8, 1, 128, 64, dtype, seed=24)
    p = c.plan()
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for lq in ([4, 4, 4], [1, 0, 3], [2, 4, 1]):
        c.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32))
        p.out.zero_()
        g.replay()
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.lq = lq
        d.check(p)


@pytest.mark.parametrize("scale_given", [False, True])
def test_drafts_with_e4m3_output(scale_given):
    c = Case([3, 4], [300, 2000], 8, 1, 128, 64, "fp8", seed=25)
    sc = torch.linspace(0.002, 0.02, 8, device="cuda") if scale_given else None
    p = c.plan(out_dtype=fp2.FP2_FP8_E4M3, out_scale=sc)
    p.run()
    c.check(p, out_scale=sc if scale_given else c.scales["v"].repeat_interleave(8))


def test_drafts_with_a_bad_page_or_factor():
    c = Case([4, 4], [900, 700], 8, 1, 128, 64, "fp8", seed=26, factors=True)
    p = c.plan()
    keep = int(c.table[0, 3])
    c.table[0, 3] = 10 ** 6
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 3)
    c.check(p, skip=(0,))
    c.table[0, 3] = keep
    c.fac["k"][1, 2, 0] = 0.0
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_INVALID_ARG, 5)
    c.check(p, skip=(1,))


def test_a_step_in_which_every_sequence_rests():
    c = Case([0, 0], [100, 40], seed=27, pad=1)
    p = c.plan(max_seqlen_q=0)
    p.out.fill_(3.0)
    p.run()
    p.check()
    assert (p.out == 3).all()
    c.cu.copy_(torch.tensor([0, 0, 1], dtype=torch.int32))  # a token above the limit of 0
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_INVALID_ARG, 1)
    assert (p.out == 3).all()


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_a_scale_of_zero_is_a_head_of_zeros(n, which):
    c = Case([n, n], [170, 40], 8, 1, 128, 16, "fp8", seed=28)
    c.scales[which][0] = 0.0
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("n", [1, 4])
def test_no_limit_on_the_keys(n):
    """max_seqlen_k as large as its type: a bound only, nothing is sized by it."""
    c = Case([n, n], [300, 40], 8, 1, 128, 64, seed=29)
    p = c.plan(max_seqlen_k=2 ** 31 - 1)
    p.run()
    c.check(p)
    c.seqlens_k[0] = 2 ** 31 - 1  # more than its pages hold
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert e.value.detail == 1
    c.check(p, skip=(0,))


def test_offsets_that_wrap_are_refused():
    """Row and key offsets whose sums pass 32 bits are bad lengths, not small ones."""
    c = Case([1, 1], [300, 40], 8, 1, 128, 0, seed=30)
    p = c.plan()
    cu_k = c.cu_k.clone()
    c.cu_k[0] = 2 ** 31 - 100
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 1)
    c.check(p, skip=(0,))
    c.cu_k.copy_(cu_k)
    c.cu.copy_(torch.tensor([2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1], dtype=torch.int32))
    p.out.fill_(3.0)
    p.run()
    with pytest.raises(fp2.Fp2Error) as e:
        p.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_INVALID_ARG, 1)
    assert (p.out == 3).all()


@pytest.mark.parametrize("dtype,Hq,Hkv,d,n", [
    ("bf16", 3, 3, 128, 1), ("bf16", 20, 5, 128, 1), ("fp8", 7, 7, 128, 2), ("fp8", 16, 16, 128, 1), ("bf16", 12, 12, 128, 1),
    ("fp8", 24, 24, 128, 1), ("bf16", 17, 17, 128, 1), ("bf16", 24, 24, 64, 1), ("bf16", 20, 10, 64, 9), ("bf16", 40, 5, 128, 3),
    ("fp8", 48, 6, 128, 4), ("fp8", 10, 5, 128, 9), ("bf16", 96, 12, 128, 3), ("fp8", 136, 17, 128, 3), ("fp8", 33, 33, 128, 1)])
@pytest.mark.parametrize("lk", [[700, 33, 3000], [40] * 30 + [900]])
def test_numbers_of_heads(dtype, Hq, Hkv, d, n, lk):
    """Heads that do not divide the CTAs, or one another."""
    c = Case([n] * len(lk), lk, Hq, Hkv, d, 16, dtype, seed=31)
    p = c.plan()
    p.run()
    c.check(p)


@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (4, "fp8"), (4, "bf16")])
def test_two_calls_at_once(n, dtype):
    """Calls on two streams, each with its own workspace, while the other runs."""
    cases = [Case([n] * 5, [4000 + 700 * i for i in range(5)], 16, 2, 128, 64, dtype, seed=32 + k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    plans = [c.plan(stream=s.cuda_stream) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p in plans:
            p.run()
    torch.cuda.synchronize()
    for c, p in zip(cases, plans):
        c.check(p)


@pytest.mark.parametrize("n", [1, 4])
def test_same_inputs_same_bits(n):
    """Shares and joins in a fixed order: a second call, alone or after others, gives the same bits."""
    c = Case([n] * 6, [10, 5000, 1, 4, 900, 2500] if n == 1 else [10, 5000, 7, 4, 900, 2500], 16, 2, 128, 16, "fp8", seed=34)
    p, other = c.plan(), Case([1], [3000], 16, 2, 128, 16, "bf16", seed=35).plan()
    p.run()
    out, lse = p.out.clone(), p.lse.clone()
    for _ in range(5):
        other.run()
        p.out.zero_()
        p.run()
        assert torch.equal(p.out.view(torch.uint8), out.view(torch.uint8)) and torch.equal(p.lse, lse)
    c.check(p)
