"""fp2_page_map against an allocator that goes request by request, and the three
serving-step calls together, as a server would run them."""
import numpy as np
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests import serve_ref as R

pytestmark = pytest.mark.gpu
OUTPUTS = ("cu_seqlens", "seqlens_k", "positions", "slot_map", "page_table", "free_head_out")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def setup(prefix, new, page, pad=0, seed=0, used=2, short=0, slack=2):
    rs = np.random.RandomState(seed)
    old = [R.pages(p, page) for p in prefix]
    after = [R.pages(p + n, page) for p, n in zip(prefix, new)]
    num = sum(after) + 5
    perm = rs.permutation(num)
    table = np.full((len(prefix), max(after) + slack), -7, np.int64)
    at = 0
    for b, n in enumerate(old):
        table[b, :n] = perm[at:at + n]
        at += n
    fresh = sum(after) - sum(old)
    free = np.concatenate([perm[:used], perm[at:at + fresh - short]])
    m = fp2.make_page_map(i32(prefix), i32(new), i32(table), i32(free), i32([used]), page_size=page, num_pages=num,
                          total_q=sum(new) + pad, max_seqlen_q=max(1, max(new)), max_seqlen_k=max(1, max(p + n for p, n in zip(prefix, new))))
    return m, table, free, used


def compare(m, want):
    for name in OUTPUTS:
        assert getattr(m, name).cpu().tolist() == want[name], name


CASES = [([0], [1], 16), ([0], [0], 16), ([5], [1], 16), ([15, 16, 17], [1, 1, 1], 16), ([0, 0, 0], [16, 17, 33], 16),
         ([63, 0, 64, 200], [0, 1, 64, 129], 64), ([0, 100000], [5000, 1], 256), ([0] * 3, [0] * 3, 32)]


@pytest.mark.parametrize("prefix,new,page", CASES)
@pytest.mark.parametrize("pad", [0, 5])
def test_small(prefix, new, page, pad):
    m, table, free, used = setup(prefix, new, page, pad)
    m.run()
    m.check()
    compare(m, R.page_map(prefix, new, table, free, used, page, sum(new) + pad))


@pytest.mark.parametrize("S,page,hi", [(511, 16, 40), (512, 64, 3), (513, 32, 70), (2000, 128, 300), (16384, 16, 20)])
def test_many_sequences(S, page, hi):
    rs = np.random.RandomState(S)
    prefix, new = rs.randint(0, 200, S).tolist(), rs.randint(0, hi, S).tolist()
    m, table, free, used = setup(prefix, new, page, 33, seed=S)
    m.run()
    m.check()
    want = R.page_map(prefix, new, table, free, used, page, sum(new) + 33)
    compare(m, want)
    m.run()  # from the same inputs the step is the same again
    m.check()
    compare(m, want)


def test_long_prompts():
    prefix, new = [0, 64, 1], [40000, 262144 - 64, 1]
    m, table, free, used = setup(prefix, new, 64)
    m.run()
    m.check()
    compare(m, R.page_map(prefix, new, table, free, used, 64, sum(new)))


def test_no_limit_on_the_keys():
    prefix, new = [10, 40, 0], [7, 30, 20]
    m, table, free, used = setup(prefix, new, 16)
    m.params.max_seqlen_k = 2 ** 31 - 1
    m.run()
    m.check()
    compare(m, R.page_map(prefix, new, table, free, used, 16, sum(new)))
    m.prefix_lens[1] = 2 ** 31 - 31  # more than a row of the table holds
    m.run()
    with pytest.raises(fp2.Fp2Error) as e:
        m.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 1)
    assert m.cu_seqlens.tolist() == [0] * 4


@pytest.mark.parametrize("what,status,detail", [
    ("new_negative", fp2.FP2_ERR_INVALID_ARG, 1), ("new_large", fp2.FP2_ERR_INVALID_ARG, 1),
    ("prefix_negative", fp2.FP2_ERR_INVALID_ARG, 1), ("keys_large", fp2.FP2_ERR_INVALID_ARG, 1),
    ("rows_short", fp2.FP2_ERR_INVALID_ARG, 1), ("free_short", fp2.FP2_ERR_DEVICE_BOUNDS, 6),
    ("head_negative", fp2.FP2_ERR_DEVICE_BOUNDS, 6), ("table_short", fp2.FP2_ERR_DEVICE_BOUNDS, 1)])
def test_errors_leave_an_empty_step(what, status, detail):
    prefix, new, page = [10, 40, 0], [7, 30, 20], 16
    m, table, free, used = setup(prefix, new, page, 4, short=1 if what == "free_short" else 0, slack=0)
    if what == "new_negative":
        m.new_lens[1] = -1
    elif what == "new_large":
        m.new_lens[1] = 31
    elif what == "prefix_negative":
        m.prefix_lens[2] = -5
    elif what == "keys_large":
        m.prefix_lens[1] = 2 ** 31 - 5
    elif what == "rows_short":
        m.params.total_q = 50
    elif what == "head_negative":
        m.free_head[0] = -1
    elif what == "table_short":
        m.params.max_seqlen_k = 2 ** 20
        m.prefix_lens[0] = 90
    m.run()
    with pytest.raises(fp2.Fp2Error) as e:
        m.check()
    assert (e.value.status, e.value.detail) == (status, detail)
    assert m.cu_seqlens.tolist() == [0] * 4 and m.seqlens_k.tolist() == m.prefix_lens.tolist()
    n = m.params.total_q
    assert m.slot_map[:n].tolist() == [-1] * n and m.positions[:n].tolist() == [0] * n
    assert m.page_table.tolist() == table.tolist() and m.free_head_out.tolist() == m.free_head.tolist()


def test_bad_page_ids_are_recorded():
    prefix, new, page = [10, 0], [3, 40], 16
    for where in ("free", "table"):
        m, table, free, used = setup(prefix, new, page)
        want = R.page_map(prefix, new, table, free, used, page, 43)
        if where == "free":
            m.free_pages[used + 1] = 10 ** 6  # the second page of sequence 1
            want["page_table"][1][1] = -1
            want["slot_map"][3 + 16:3 + 32] = [-1] * 16
        else:
            m.page_table[0, 0] = -3
            want["page_table"][0][0] = -3
            want["slot_map"][:3] = [-1] * 3
        m.run()
        with pytest.raises(fp2.Fp2Error) as e:
            m.check()
        assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 3)
        compare(m, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_served_batch(dtype, captured):
    """Map, append and decode step after step from one pool of pages: a ragged
    first step of up to 16 tokens, then single tokens (one request rests, one
    drafts 3), each step's attention checked against 64 bits over all the rows
    that were appended so far, read back from the requests' own history."""
    Hq, Hkv, d, page, S, T = 8, 2, 128, 16, 4, 24
    fp8 = dtype == "fp8"
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    steps = [[16, 3, 1, 4], [1, 1, 0, 1], [1, 1, 1, 3], [1, 1, 1, 1], [0, 1, 5, 1]]
    maxk, npages = 64, 40
    rs = np.random.RandomState(7)
    g = torch.Generator("cuda").manual_seed(7)
    free = i32(rs.permutation(npages))
    lens, heads = [i32([0] * S), i32([0] * S)], [i32([0]), i32([0])]
    table = i32(np.full((S, maxk // page), -1))
    new = i32([0] * S)
    rows = torch.zeros((T, (Hq + 2 * Hkv) * d), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.view(T, h, d) for x, h in zip(rows.split([Hq * d, Hkv * d, Hkv * d], 1), (Hq, Hkv, Hkv)))
    kc, vc = (torch.full((npages, page, Hkv, d), float("nan"), device="cuda").to(kind) for _ in "kv")
    sc = {n: (0.01 + 0.002 * torch.rand(h, generator=g, device="cuda")) if fp8 else None for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    scales = {n + "_scale": sc[n] for n in "qkv"}
    w = {n: 1 + 0.1 * torch.randn(d, generator=g, device="cuda") for n in "qk"}
    inv = (1.0 / 10000.0 ** (torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    dt = fp2.FP2_FP8_E4M3 if fp8 else fp2.FP2_BF16
    ops = []
    ws = None
    for at in range(2):  # the lengths and the head swap their buffers from step to step
        m = fp2.make_page_map(lens[at], new, table, free, heads[at], page_size=page, num_pages=npages, total_q=T, max_seqlen_q=16,
                              max_seqlen_k=maxk, seqlens_k=lens[1 - at], free_head_out=heads[1 - at], workspace=ws)
        a = fp2.make_append(q, k, v, kc, vc, m.positions, m.slot_map, dtype=dt, inv_freq=inv, q_weight=w["q"], k_weight=w["k"], **scales)
        D = fp2.make_decode(a.q_out, kc, vc, m.cu_seqlens, Hq=Hq, Hkv=Hkv, d=d, dtype=dt, max_seqlen_q=16, max_seqlen_k=maxk,
                            seqlens_k=m.seqlens_k, page_table=table, page_size=page, with_lse=True, **scales)
        ops.append((m, a, D))
    run = [lambda ops=o: [x.run() for x in ops] for o in ops]
    if captured:
        graphs = []
        for f in run:
            f()
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                f()
            graphs.append(gr)
        run = [gr.replay for gr in graphs]
        for x in lens + heads:  # the warm-up steps were empty; start anew all the same
            x.zero_()
    history = [[np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))] for _ in range(S)]
    for n, fresh in enumerate(steps):
        new.copy_(i32(fresh))
        rows.copy_(torch.randn(rows.shape, generator=g, device="cuda").bfloat16())
        m, a, D = ops[n % 2]
        run[n % 2]()
        for x in (m, a, D):
            x.check()
        at = np.concatenate([[0], np.cumsum(fresh)])
        assert m.cu_seqlens.tolist() == at.tolist()
        for b in range(S):
            sl = slice(at[b], at[b + 1])
            pos = len(history[b][0]) + np.arange(fresh[b])
            assert m.positions[sl].tolist() == pos.tolist()
            qr, qt = R.append_rows(q[sl].double().cpu().numpy(), w["q"].double().cpu().numpy(), 1e-6, pos, inv.cpu().numpy(), d, False,
                                   1.0, sc["q"].double().cpu().numpy() if fp8 else None, kind)
            kr, kt = R.append_rows(k[sl].double().cpu().numpy(), w["k"].double().cpu().numpy(), 1e-6, pos, inv.cpu().numpy(), d, False,
                                   1.0, sc["k"].double().cpu().numpy() if fp8 else None, kind)
            # what was stored is within its rounding; the attention is then
            # checked on the stored values, of which the request keeps a copy
            slots = m.slot_map[sl].long()
            flat = [x.view(-1, Hkv, d).view(torch.uint8)[slots].view(kind) if fp8 else x.view(-1, Hkv, d)[slots] for x in (kc, vc)]
            assert (np.abs(flat[0].double().cpu().numpy() - kr) <= kt).all()
            assert (np.abs(a.q_out[sl].double().cpu().numpy() - qr) <= qt).all()
            un = [1.0 if not fp8 else sc[x].double().cpu().numpy()[:, None] for x in "kv"]
            history[b] = [np.concatenate([h, x.double().cpu().numpy() * u]) for h, x, u in zip(history[b], flat, un)]
            if not fresh[b]:
                continue
            qd = a.q_out[sl].double() * (sc["q"].double()[:, None] if fp8 else 1.0)
            K, V = (torch.tensor(h, device="cuda") for h in history[b])
            ref, lse, absv, dot = R.decode(qd, K, V, Hq // Hkv)
            tol, tol_lse = R.decode_bounds(ref, absv, dot, len(K), d, dtype, torch.bfloat16)
            assert ((D.out[sl].double() - ref).abs() <= tol).all()
            assert ((D.lse[sl].double() - lse).abs() <= tol_lse).all()
