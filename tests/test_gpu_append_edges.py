"""fp2_append with scales of 0, and the caches it leaves behind read by fp2_decode."""
import pytest
import torch

from block_sparse_long_blockmean_b200 import fp2
from tests import serve_ref as R
from tests.test_gpu_append import freqs

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "v", "qkv"])
def test_a_scale_of_zero_stores_zeros(which, norm):
    """A head of zeros has an absmax scale of 0: zeros are stored for it and the others as they
    are, and decoding from that cache gives the attention of a head of zeros."""
    T, Hq, Hkv, d = 40, 8, 2, 128
    g = torch.Generator("cuda").manual_seed(5)
    x = {n: torch.randn((T, h, d), generator=g, device="cuda").bfloat16() for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    sc = {n: 0.01 * (1 + torch.rand(h, generator=g, device="cuda")) for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    for n in which:
        x[n][:, 1] = 0
        sc[n][1] = 0
    w = torch.ones(d, device="cuda") if norm else None
    kc, vc = (torch.full((T, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in "kv")
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    scales = {n + "_scale": s for n, s in sc.items()}
    a = fp2.make_append(x["q"], x["k"], x["v"], kc, vc, pos, slots, dtype=fp2.FP2_FP8_E4M3, inv_freq=freqs(d), q_weight=w, k_weight=w, **scales)
    a.run()
    a.check()
    got = {"q": a.q_out, "k": kc, "v": vc}
    for n in "qkv":
        src, unit = x[n].double().cpu().numpy(), sc[n].double().cpu().numpy()
        live = [h for h in range(src.shape[1]) if unit[h]]
        ref, tol = R.append_rows(src[:, live], w.double().cpu().numpy() if norm and n != "v" else None, 1e-6, pos.cpu().numpy(), freqs(d).cpu().numpy(),
                                 d if n != "v" else 0, False, 1.0, unit[live], E4M3)
        y = got[n].double().cpu().numpy()
        assert (abs(y[:, live] - ref) <= tol).all()
        if n in which:
            assert (y[:, 1] == 0).all()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    p = fp2.make_decode(a.q_out[T - 1:], kc, vc, cu, Hq=Hq, Hkv=Hkv, d=d, dtype=fp2.FP2_FP8_E4M3, max_seqlen_q=1, max_seqlen_k=T,
                        seqlens_k=torch.tensor([T], dtype=torch.int32, device="cuda"),
                        cu_seqlens_k=torch.tensor([0, T], dtype=torch.int32, device="cuda"), with_lse=True, **scales)
    p.run()
    p.check()
    q, K, V = (got[n].double() * sc[n].double()[:, None] for n in "qkv")
    ref, lse, absv, dot = R.decode(q[T - 1:], K, V, Hq // Hkv)
    tol, tol_lse = R.decode_bounds(ref, absv, dot, T, d, "fp8", torch.bfloat16)
    assert ((p.out.double() - ref).abs() <= tol).all() and ((p.lse.double() - lse).abs() <= tol_lse).all()
