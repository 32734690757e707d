"""The serving step's calls, each for the first time in its process inside a stream
capture: nothing they set up on the way may need a synchronising call."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
from block_sparse_long_blockmean_b200 import fp2
E4M3 = torch.float8_e4m3fn
dtype, n, S, Hq, Hkv, d, page, pages = {dtype!r}, {n}, 3, 8, 1, 128, 64, 20
fp8 = dtype == "fp8"
code, kind, dev = (fp2.FP2_FP8_E4M3 if fp8 else fp2.FP2_BF16), (E4M3 if fp8 else torch.bfloat16), "cuda"
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
T = S * n
prefix, new, free, head = i32(*[100, 30, 70]), i32(*[n] * S), torch.arange(pages, dtype=torch.int32, device=dev), i32(6)
table = torch.full((S, 4), -1, dtype=torch.int32, device=dev)
table[0, :2], table[1, :1], table[2, :2] = i32(0, 1), i32(2), i32(3, 4)
g = torch.Generator("cuda").manual_seed(1)
q, k, v = (torch.randn((T, h, d), generator=g, device=dev).bfloat16() for h in (Hq, Hkv, Hkv))
kc, vc = (torch.randn((pages, page, Hkv, d), generator=g, device=dev).to(kind) for _ in "kv")
sc = {{x + "_scale": torch.full((h,), 0.01, device=dev) for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}} if fp8 else {{}}
freq = torch.linspace(0.01, 1, d // 2, device=dev)
m = fp2.make_page_map(prefix, new, table, free, head, page_size=page, num_pages=pages, total_q=T, max_seqlen_q=n, max_seqlen_k=200)
a = fp2.make_append(q, k, v, kc, vc, m.positions, m.slot_map, dtype=code, inv_freq=freq, **sc)
p = fp2.make_decode(a.q_out, kc, vc, m.cu_seqlens, Hq=Hq, Hkv=Hkv, d=d, dtype=code, max_seqlen_q=n, max_seqlen_k=200,
                    seqlens_k=m.seqlens_k, page_table=table, page_size=page, with_lse=True, **sc)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for x in (m, a, p):
        x.run()
graph.replay()
for x in (m, a, p):
    x.check()
out, lse = p.out.clone(), p.lse.clone()
p.out.zero_()
table[:, 2:] = -1
for x in (m, a, p):
    x.run()
    x.check()
assert torch.isfinite(out.float()).all() and torch.equal(p.out, out) and torch.equal(p.lse, lse)
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("fp8", 1), ("bf16", 4), ("fp8", 4)])
def test_first_calls_inside_a_capture(dtype, n):
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(dtype=dtype, n=n)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
