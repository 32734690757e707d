"""Plain 64-bit forms of the serving-step calls (fp2_page_map, fp2_append,
fp2_decode) and the error bounds their tests use, derived from the arithmetic
the calls promise: fp32 (or wider) inside, one rounding at the end.

A rounding to a type with spacing eps is off by at most eps / 2 of the value:
bf16 2^-8, e4m3 2^-4 (and 2^-10 of its unit below its smallest normal)."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
SUBNORMAL = {torch.bfloat16: 0.0, torch.float8_e4m3fn: 2.0 ** -10}


def pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------- map ----

def page_map(prefix, new, table, free, head, page, total_q):
    """Request by request, as an allocator would."""
    table = np.array(table, np.int64)
    cu, pos, slots = [0], [], []
    for b, (p, n) in enumerate(zip(prefix, new)):
        for k in range(pages(p, page), pages(p + n, page)):
            table[b, k] = free[head]
            head += 1
        for t in range(p, p + n):
            pos.append(t)
            slots.append(int(table[b, t // page]) * page + t % page)
        cu.append(cu[-1] + n)
    pad = total_q - cu[-1]
    return dict(cu_seqlens=cu, seqlens_k=[p + n for p, n in zip(prefix, new)], positions=pos + [0] * pad,
                slot_map=slots + [-1] * pad, page_table=table.tolist(), free_head_out=[head])


# ---------------------------------------------------------------- append ----

def turned(x, positions, inv_freq, rot, interleaved, scale):
    """x [T, heads, d] (float64) rotated; angles in extended precision."""
    x = x.copy()
    if rot == 0:
        return x
    ang = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None]
    c = (np.cos(ang) * scale).astype(np.float64)[:, None]
    s = (np.sin(ang) * scale).astype(np.float64)[:, None]
    one = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    two = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., one].copy(), x[..., two].copy()
    x[..., one] = a * c - b * s
    x[..., two] = b * c + a * s
    return x


def normed(x, w, eps):
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def append_rows(x, w, eps, positions, inv_freq, rot, interleaved, scale, unit, out_type):
    """(value, bound) of the stored rows.  Besides the last rounding: the norm's
    sum, rsqrt and products are off by under 2^-20 relative (a sum of at most 128
    squares pairwise over lanes, 16 roundings of 2^-24 in sequence, rsqrt 2^-22),
    cos and sin by under 2^-21 absolute (the turn is rounded to a float, 2 pi 2^-25,
    and the function is good to 2^-23), so a pair's members by 2^-19 (|a| + |b|)."""
    y = normed(x, w, eps)
    z = turned(y, positions, inv_freq, rot, interleaved, scale)
    size = np.abs(y).copy()
    if rot:
        one = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        two = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        both = (np.abs(y[..., one]) + np.abs(y[..., two])) * max(1.0, abs(scale))
        size[..., one] = both
        size[..., two] = both
    if unit is not None:
        z, size = z / unit[:, None], size / unit[:, None]
        z = np.clip(z, -448, 448)
    return z, HALF[out_type] * np.abs(z) + SUBNORMAL[out_type] + 2.0 ** -19 * size * (1 + HALF[out_type])


# ---------------------------------------------------------------- decode ----

def decode(q, K, V, G):
    """q [Lq, Hq, d], K and V [Lk, Hkv, d] in float64 (dequantised): out, lse and
    what their errors scale with: sum p|v| and the largest sum |q k| / sqrt(d)."""
    Lq, Hq, d = q.shape
    Lk = K.shape[0]
    out = torch.zeros((Lq, Hq, d), dtype=torch.float64, device=q.device)
    absv, lse = torch.zeros_like(out), torch.zeros((Lq, Hq), dtype=torch.float64, device=q.device)
    dot = torch.zeros_like(lse)
    for t in range(Lq):
        n = Lk - Lq + t + 1  # keys that row t sees; the others are never touched
        for h in range(Hq):
            k, v = K[:n, h // G], V[:n, h // G]
            z = (k @ q[t, h]) / math.sqrt(d)
            p = torch.softmax(z, 0)
            out[t, h], absv[t, h] = p @ v, p @ v.abs()
            lse[t, h] = torch.logsumexp(z, 0)
            dot[t, h] = (k.abs() @ q[t, h].abs()).max() / math.sqrt(d)
    return out, lse, absv, dot


def decode_bounds(ref, absv, dot, Lk, d, dtype, out_type, unit=None):
    """Bounds of |out - ref| and |lse - ref|.  A logit is a sum of d products in
    fp32, each addition off by at most 2^-22 of the terms so far (a tensor core
    may truncate): dz = d 2^-22 sum|q k| / sqrt(d).  Weights e^z are then off by
    dz relative, both in the sum and in the total; exp2 by 2^-21; a weight is
    rounded once more for the product with v: to two bf16 terms (2^-16) or to
    fp16 (2^-11); the sums over keys add at most Lk / 16 + 64 terms in sequence."""
    dz = d * 2.0 ** -22 * dot
    weight = 2.0 ** -11 if dtype == "fp8" else 2.0 ** -16
    sums = (Lk / 16 + 64) * 2.0 ** -22
    inner = absv * (2 * dz[..., None] + weight + 2.0 ** -20 + 2 * sums)
    if unit is not None:
        ref, inner = ref / unit[:, None], inner / unit[:, None]
    out = HALF[out_type] * (ref.abs() + inner) + SUBNORMAL[out_type] + inner
    return out, dz + sums + 2.0 ** -20
