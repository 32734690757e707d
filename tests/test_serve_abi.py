"""Host side of fp2_page_map, fp2_append and fp2_decode, without a GPU: struct
layout, workspace sizes, and the status codes of calls that are refused before
any CUDA work (the pointers below are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest
import torch

from block_sparse_long_blockmean_b200 import build as B
from block_sparse_long_blockmean_b200 import fp2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = fp2.FP2_OK, fp2.FP2_ERR_INVALID_ARG, fp2.FP2_ERR_UNSUPPORTED, fp2.FP2_ERR_WORKSPACE
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B.build()
    return fp2.lib()


def params(**kw):
    P = fp2.Params()
    P.num_seqs, P.num_q_heads, P.num_kv_heads, P.head_dim = 4, 8, 2, 128
    P.total_q, P.max_seqlen_q, P.max_seqlen_k = 4, 1, 1000
    P.page_size, P.max_pages_per_seq, P.num_pages = 64, 16, 100
    P.workspace, P.workspace_bytes = 1 << 40, 1 << 30
    for k, v in kw.items():
        setattr(P, k, v)
    return P


def test_append_io_layout_matches_the_header(tmp_path):
    fields = [f for f, _ in fp2.AppendIO._fields_]
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "fp2.h"', "int main(void){",
            'printf("%zu\\n%d\\n", sizeof(fp2_append_io), FP2_DECODE_MAX_Q);']
    prog += [f'printf("%zu\\n", offsetof(fp2_append_io, {f}));' for f in fields] + ["return 0;}"]
    c, exe = tmp_path / "probe.c", tmp_path / "probe"
    c.write_text("\n".join(prog))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(fp2.AppendIO), fp2.FP2_DECODE_MAX_Q] + [getattr(fp2.AppendIO, f).offset for f in fields]


# ------------------------------------------------------------------- map ----

def call_map(lib, P, n_free=50, **at):
    names = ["prefix_lens", "new_lens", "free_pages", "free_head", "page_table", "cu_seqlens", "seqlens_k", "positions", "slot_map",
             "free_head_out"]
    a = {n: MB * (i + 1) for i, n in enumerate(names)}
    a.update(at)
    return lib.fp2_page_map(a["prefix_lens"], a["new_lens"], a["free_pages"], n_free, a["free_head"], a["page_table"], a["cu_seqlens"],
                            a["seqlens_k"], a["positions"], a["slot_map"], a["free_head_out"], ctypes.byref(P) if P else None)


@pytest.mark.parametrize("field,value,code", [
    ("num_seqs", 0, INVALID), ("num_seqs", 16385, UNSUPPORTED), ("total_q", -1, INVALID), ("max_pages_per_seq", 0, INVALID),
    ("page_size", 48, UNSUPPORTED), ("page_size", 8, UNSUPPORTED), ("page_size", 512, UNSUPPORTED), ("page_size", 0, UNSUPPORTED),
    ("num_pages", 0, INVALID), ("num_pages", 1 << 25, UNSUPPORTED), ("max_seqlen_q", -1, INVALID), ("max_seqlen_k", 0, INVALID),
    ("workspace", None, WORKSPACE), ("workspace", (1 << 40) + 8, WORKSPACE), ("workspace_bytes", 255, WORKSPACE)])
def test_map_refuses_sizes(lib, field, value, code):
    assert call_map(lib, params(**{field: value})) == code


def test_map_refuses_pointers(lib):
    P = params()
    assert call_map(lib, None) == INVALID
    for n in ("prefix_lens", "new_lens", "free_pages", "free_head", "page_table", "cu_seqlens", "seqlens_k", "positions", "slot_map",
              "free_head_out"):
        assert call_map(lib, P, **{n: None}) == INVALID, n
        assert call_map(lib, P, **{n: MB * 40 + 2}) == INVALID, n
    assert call_map(lib, P, n_free=-1) == INVALID
    # outputs on inputs or on each other
    assert call_map(lib, P, seqlens_k=MB) == INVALID            # = prefix_lens
    assert call_map(lib, P, seqlens_k=MB + 12) == INVALID       # its last entry
    assert call_map(lib, P, free_head_out=MB * 4) == INVALID    # = free_head
    assert call_map(lib, P, slot_map=MB * 8) == INVALID         # = positions
    assert call_map(lib, P, page_table=MB * 3 - 4) == INVALID   # reaches into free_pages


# ---------------------------------------------------------------- append ----

def append_io(**kw):
    io = fp2.AppendIO()
    for i, n in enumerate(["q", "k", "v", "q_weight", "k_weight", "inv_freq", "positions", "slot_map", "q_out", "k_cache", "v_cache"]):
        setattr(io, n, (1 << 32) * (i + 1))
    io.q_stride, io.k_stride, io.v_stride = 1536, 1536, 1536
    io.eps, io.rope_scale, io.rotary_dim = 1e-6, 1.0, 128
    for k, v in kw.items():
        setattr(io, k, v)
    return io


def call_append(lib, io, P, dtype=fp2.FP2_BF16):
    return lib.fp2_append(ctypes.byref(io) if io else None, dtype, ctypes.byref(P) if P else None)


@pytest.mark.parametrize("field,value,code", [
    ("num_kv_heads", 3, INVALID), ("num_q_heads", 6, UNSUPPORTED), ("num_q_heads", 32, UNSUPPORTED), ("head_dim", 96, UNSUPPORTED),
    ("total_q", -1, INVALID), ("page_size", 24, UNSUPPORTED), ("num_pages", 0, INVALID), ("workspace_bytes", 0, WORKSPACE),
    ("k_block_factor", MB, UNSUPPORTED), ("v_block_factor", MB, UNSUPPORTED)])
def test_append_refuses_sizes(lib, field, value, code):
    assert call_append(lib, append_io(), params(**{field: value})) == code


@pytest.mark.parametrize("field,value,code", [
    ("rotary_dim", -8, INVALID), ("rotary_dim", 136, INVALID), ("rotary_dim", 12, UNSUPPORTED), ("eps", -1.0, INVALID),
    ("eps", float("nan"), INVALID), ("eps", float("inf"), INVALID), ("rope_scale", float("nan"), INVALID), ("interleaved", 2, INVALID),
    ("inv_freq", None, INVALID), ("positions", None, INVALID), ("slot_map", None, INVALID), ("q", None, INVALID), ("k", None, INVALID),
    ("v", None, INVALID), ("q_out", None, INVALID), ("k_cache", None, INVALID), ("v_cache", None, INVALID), ("q_stride", 1020, INVALID),
    ("k_stride", 252, INVALID), ("v_stride", 257, INVALID), ("q", (1 << 32) + 4, INVALID), ("q_weight", (4 << 32) + 8, INVALID), ("k_weight", (5 << 32) + 4, INVALID),
    ("inv_freq", (6 << 32) + 2, INVALID), ("positions", (7 << 32) + 1, INVALID), ("slot_map", (8 << 32) + 2, INVALID), ("q_out", (9 << 32) + 8, INVALID),
    ("k_cache", (10 << 32) + 8, INVALID), ("k_cache", 11 << 32, INVALID), ("v_cache", (1 << 32) + 1024, INVALID), ("q_out", 1 << 32, INVALID)])
def test_append_refuses_io(lib, field, value, code):
    assert call_append(lib, append_io(**{field: value}), params()) == code


def test_append_other_refusals(lib):
    assert call_append(lib, None, params()) == INVALID
    assert call_append(lib, append_io(), None) == INVALID
    assert call_append(lib, append_io(), params(), 2) == INVALID
    assert call_append(lib, append_io(), params(), fp2.FP2_FP8_E4M3) == INVALID  # no scales
    assert call_append(lib, append_io(), params(total_q=0)) == OK                # nothing to do


# ---------------------------------------------------------------- decode ----

def call_decode(lib, P, block=128, dtype=fp2.FP2_BF16, table=MB, cu=2 * MB, q=1 << 32, k=2 << 32, v=3 << 32, out=4 << 32, lse=5 << 32):
    return lib.fp2_decode(q, k, v, table, cu, block, dtype, out, lse, ctypes.byref(P) if P else None)


@pytest.mark.parametrize("field,value,code", [
    ("num_seqs", 0, INVALID), ("num_kv_heads", 3, INVALID), ("num_q_heads", 6, UNSUPPORTED), ("num_q_heads", 32, UNSUPPORTED),
    ("head_dim", 80, UNSUPPORTED), ("max_seqlen_q", 17, UNSUPPORTED), ("max_seqlen_q", -1, INVALID), ("max_seqlen_k", 0, INVALID),
    ("total_q", -1, INVALID)])
def test_decode_refuses_sizes(lib, field, value, code):
    P = params(**{field: value})
    assert call_decode(lib, P) == code
    assert fp2.decode_workspace_size(P) == 0 or field == "max_seqlen_q" and value == 17 and fp2.decode_workspace_size(P) == 0


@pytest.mark.parametrize("field,value,code", [
    ("page_size", 40, UNSUPPORTED), ("num_pages", 0, INVALID), ("num_pages", 1 << 26, UNSUPPORTED), ("max_pages_per_seq", 0, INVALID),
    ("workspace", None, WORKSPACE), ("workspace", (1 << 40) + 16, WORKSPACE), ("out_dtype", 3, INVALID),
    ("out_dtype", fp2.FP2_FP8_E4M3, INVALID), ("k_block_factor", MB, INVALID)])
def test_decode_refuses_the_rest(lib, field, value, code):
    assert call_decode(lib, params(**{field: value})) == code


def test_decode_refuses_pointers_types_and_blocks(lib):
    P = params()
    assert call_decode(lib, None) == INVALID
    for n in ("q", "k", "v", "out", "cu"):
        assert call_decode(lib, P, **{n: None}) == INVALID
    for n in ("q", "k", "v", "out"):
        assert call_decode(lib, P, **{n: (7 << 32) + 8}) == INVALID
    assert call_decode(lib, P, lse=(7 << 32) + 2) == INVALID
    assert call_decode(lib, P, block=96) == UNSUPPORTED
    assert call_decode(lib, P, dtype=5) == INVALID
    scales = dict(q_scale=MB, k_scale=MB, v_scale=MB)
    assert call_decode(lib, P, dtype=fp2.FP2_FP8_E4M3) == INVALID
    assert call_decode(lib, params(head_dim=64, **scales), dtype=fp2.FP2_FP8_E4M3) == UNSUPPORTED
    assert call_decode(lib, params(**scales), block=64, dtype=fp2.FP2_FP8_E4M3) == UNSUPPORTED
    assert call_decode(lib, params(k_block_factor=MB, **scales), dtype=fp2.FP2_FP8_E4M3) == INVALID
    need = fp2.decode_workspace_size(P)
    assert need > 256 and call_decode(lib, params(workspace_bytes=need - 1)) == WORKSPACE
    assert call_decode(lib, params(total_q=0)) == OK
    assert call_decode(lib, params(total_k=0), table=None) == INVALID


def test_decode_refuses_outputs_over_inputs(lib):
    P = params()
    q, k, v, out = (n << 32 for n in (1, 2, 3, 4))
    nq = P.total_q * P.num_q_heads * P.head_dim * 2
    nc = P.num_pages * P.page_size * P.num_kv_heads * P.head_dim * 2
    for at in (q, q + nq - 16, q - nq + 16, k, k + nc - 16, v, v - nq + 16):
        assert call_decode(lib, P, out=at) == INVALID
    nl = P.total_q * P.num_q_heads * 4
    for at in (q, q + nq - 4, q - nl + 4, k + 64, v + nc - 4, out, out + nq - 4, out - nl + 4):
        assert call_decode(lib, P, lse=at) == INVALID


# --------------------------------------------------- the Python handles' ----

def test_handles_refuse_what_the_abi_cannot_see():
    """Types, shapes, layouts and devices are refused before anything is allocated."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kw = dict(page_size=16, num_pages=10, total_q=4, max_seqlen_q=4, max_seqlen_k=40)
    with pytest.raises(TypeError):
        fp2.make_page_map(i(3).long(), i(3), i(3, 4), i(9), i(1), **kw)
    with pytest.raises(ValueError):
        fp2.make_page_map(i(3), i(2), i(3, 4), i(9), i(1), **kw)
    with pytest.raises(ValueError):
        fp2.make_page_map(i(3), i(3), i(4, 3).t(), i(9), i(1), **kw)
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for q, k, kc, err in ((h(4, 8, 128).float(), h(4, 2, 128), h(5, 16, 2, 128), TypeError),
                          (h(4, 8, 128), h(3, 2, 128), h(5, 16, 2, 128), ValueError),
                          (h(8, 4, 128).transpose(0, 1), h(4, 2, 128), h(5, 16, 2, 128), ValueError),
                          (h(4, 8, 128), h(4, 2, 128), h(5, 16, 4, 128), ValueError)):
        with pytest.raises(err):
            fp2.make_append(q, k, k, kc, kc.clone(), i(4), i(4), dtype=fp2.FP2_BF16)
    dec = dict(Hq=8, Hkv=2, d=128, dtype=fp2.FP2_BF16, max_seqlen_q=1, max_seqlen_k=64)
    with pytest.raises(ValueError):
        fp2.make_decode(h(4, 8, 64), h(64, 2, 128), h(64, 2, 128), i(5), **dec)
    with pytest.raises(TypeError):
        fp2.make_decode(h(4, 8, 128), h(64, 2, 128), h(64, 2, 128).float(), i(5), **dec)
    with pytest.raises(ValueError):
        fp2.make_decode(h(4, 8, 128), h(4, 16, 2, 128), h(4, 16, 2, 128), i(5), page_table=i(4, 3), page_size=32, **dec)


def test_handles_refuse_other_workspaces():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kw = dict(page_size=16, num_pages=10, total_q=4, max_seqlen_q=4, max_seqlen_k=40)
    args = (i(3), i(3), i(3, 4), i(9), i(1))
    with pytest.raises(TypeError):
        fp2.make_page_map(*args, workspace=torch.zeros(256), **kw)
    with pytest.raises(ValueError):
        fp2.make_page_map(*args, workspace=torch.zeros(1, dtype=torch.uint8).expand(256), **kw)
    with pytest.raises(ValueError):
        fp2.make_page_map(*args, workspace=torch.zeros(256, dtype=torch.uint8, device="meta"), **kw)
