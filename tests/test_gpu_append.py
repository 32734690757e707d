"""fp2_append against the plain 64-bit form: norms, both pairings, partial
rotations, far positions, types, head layouts, strides, slots, errors."""
import numpy as np
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests import serve_ref as R

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def freqs(rot, theta=10000.0):
    return (1.0 / theta ** (torch.arange(0, rot, 2, dtype=torch.float64) / max(1, rot))).float().cuda()


def run_case(T, Hq, Hkv, d, rot, inter=False, dtype="bf16", norm="qk", page=64, fused=True, pos=None, seed=0, size=1.0, scale=1.0,
             eps=1e-6, skip=(), spare=1):
    g = torch.Generator("cuda").manual_seed(seed)
    rs = np.random.RandomState(seed)
    width = (Hq + 2 * Hkv) * d
    if fused:
        rows = (size * torch.randn((T, width), generator=g, device="cuda")).bfloat16()
        q, k, v = (x.view(T, h, d) for x, h in zip(rows.split([Hq * d, Hkv * d, Hkv * d], 1), (Hq, Hkv, Hkv)))
    else:
        q, k, v = ((size * torch.randn((T, h, d), generator=g, device="cuda")).bfloat16() for h in (Hq, Hkv, Hkv))
    w = {n: 1 + 0.3 * torch.randn(d, generator=g, device="cuda") if n in norm else None for n in "qk"}
    f = freqs(rot) if rot else None
    pos = rs.randint(0, 300000, T) if pos is None else np.asarray(pos)
    npg = R.pages(T, page or 1) + spare
    n_rows = npg * page if page else T + spare
    slots = rs.permutation(n_rows)[:T].astype(np.int32)
    slots[list(skip)] = -1
    kind = E4M3 if dtype == "fp8" else torch.bfloat16
    shape = (npg, page, Hkv, d) if page else (n_rows, Hkv, d)
    kc, vc = (torch.full(shape, 5.0, device="cuda").to(kind) for _ in "kv")
    sc = {n: (0.005 * (1 + torch.rand(h, generator=g, device="cuda")) if dtype == "fp8" else None) for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    a = fp2.make_append(q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(slots).cuda(),
                        dtype=fp2.FP2_FP8_E4M3 if dtype == "fp8" else fp2.FP2_BF16, inv_freq=f, interleaved=inter, q_weight=w["q"],
                        k_weight=w["k"], eps=eps, rope_scale=scale, q_scale=sc["q"], k_scale=sc["k"], v_scale=sc["v"])
    src = {n: x.double().cpu().numpy() for n, x in (("q", q), ("k", k), ("v", v))}
    a.run()
    a.check()
    fr = f.cpu().numpy() if rot else None
    live = slots >= 0
    for n, got in (("q", a.q_out), ("k", kc), ("v", vc)):
        unit = sc[n].double().cpu().numpy() if sc[n] is not None else None
        wn = w[n].double().cpu().numpy() if n != "v" and w[n] is not None else None
        ref, tol = R.append_rows(src[n], wn, eps, pos, fr, rot if n != "v" else 0, inter, scale if n != "v" else 1.0, unit, kind)
        got = got.double().cpu().numpy()
        if n != "q":
            got = got.reshape(n_rows, Hkv, d)
            rest = np.ones(n_rows, bool)
            rest[slots[live]] = False
            assert (got[rest] == float(torch.tensor(5.0).to(kind).float())).all(), "rows without a token were written"
            got, ref, tol = got[slots[live]], ref[live], tol[live]
        off = np.abs(got - ref) / np.maximum(tol, 1e-300)
        assert np.isfinite(got).all() and off.max() <= 1, (n, off.max())
    return a


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (1, 1, 128), (8, 2, 128), (5, 5, 64), (32, 8, 128)])
@pytest.mark.parametrize("T", [1, 7, 33])
@pytest.mark.parametrize("inter", [False, True])
def test_shapes(Hq, Hkv, d, T, inter):
    run_case(T, Hq, Hkv, d, d, inter, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rot", [0, 8, 24, 32, 64, 104, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_partial_rotation(dtype, rot, inter):
    run_case(19, 8, 2, 128, rot, inter, dtype, seed=2)


@pytest.mark.parametrize("norm", ["", "q", "k", "qk"])
@pytest.mark.parametrize("page", [0, 16, 256])
@pytest.mark.parametrize("fused", [False, True])
def test_norms_layouts_and_strides(norm, page, fused):
    run_case(45, 8, 2, 64, 64, False, norm=norm, page=page, fused=fused, seed=3, skip=(0, 7, 44))


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(inter):
    """Angles of far positions keep their fraction of a turn: a float's position
    times frequency would be off by up to 60 radians at 2^30."""
    run_case(12, 4, 2, 128, 128, inter, pos=[0, 1, 131071, 262143, 2 ** 20, 2 ** 24 - 1, 2 ** 24 + 1, 2 ** 27 + 3, 2 ** 29 + 1,
                                             2 ** 30 + 1, 999999937, 16777259], seed=4)


def test_large_and_tiny_values():
    run_case(9, 4, 2, 128, 128, size=200.0, seed=5)
    run_case(9, 4, 2, 128, 128, size=1e-4, seed=6)
    run_case(9, 4, 2, 128, 128, size=40.0, dtype="fp8", norm="", seed=7)  # saturates
    run_case(9, 4, 2, 128, 64, size=1.0, scale=1.2079, seed=8)


def test_many_tokens():
    run_case(3001, 4, 2, 64, 64, seed=9)
    run_case(1111, 8, 1, 128, 128, True, "fp8", seed=10)


def test_in_place_queries():
    T, Hq, Hkv, d = 37, 8, 2, 128
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    caches = [torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pos, slots = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2))
    w = torch.ones(d, device="cuda")
    kw = dict(dtype=fp2.FP2_BF16, inv_freq=freqs(d), q_weight=w, k_weight=w)
    a = fp2.make_append(q, k, v, caches[0], caches[1], pos, slots, **kw)
    a.run()
    mine = q.clone()
    b = fp2.make_append(mine, k, v, caches[2], caches[3], pos, slots, q_out=mine, **kw)
    b.run()
    a.check(), b.check()
    assert torch.equal(a.q_out, mine) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_slot_outside_the_cache_is_recorded():
    T, d = 4, 128
    q, k, v = (torch.randn((T, h, d), device="cuda").bfloat16() for h in (4, 2, 2))
    kc, vc = (torch.full((1, 16, 2, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 16, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    a = fp2.make_append(q, k, v, kc, vc, pos, slots, dtype=fp2.FP2_BF16, inv_freq=freqs(d))
    a.run()
    with pytest.raises(fp2.Fp2Error) as e:
        a.check()
    assert (e.value.status, e.value.detail) == (fp2.FP2_ERR_DEVICE_BOUNDS, 7)
    assert torch.equal(vc[0, 3], v[0])
    rest = [i for i in range(16) if i != 3]
    assert (kc[0, rest] == 3).all() and (vc[0, rest] == 3).all()
    a.run()  # the error word is clear again after check()
    slots.copy_(torch.arange(4))
    with pytest.raises(fp2.Fp2Error):
        a.check()
    a.run()
    a.check()


def test_graph_replay_reads_the_buffers():
    T, d = 5, 128
    q, k, v = (torch.randn((T, h, d), device="cuda").bfloat16() for h in (4, 2, 2))
    kc, vc = (torch.zeros((64, 2, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pos, slots = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2))
    a = fp2.make_append(q, k, v, kc, vc, pos, slots, dtype=fp2.FP2_BF16, inv_freq=freqs(d))
    a.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    slots.add_(20)
    v.neg_()
    g.replay()
    a.check()
    assert torch.equal(vc[20:25], v) and torch.equal(vc[:5], -v)
