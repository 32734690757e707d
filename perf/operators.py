"""The serving-step operators that are measured: the page map, the norm + rotation + cache append, and
the decode attention over the cache, in their plain form (torch operations) and as the library's calls.

A case is a dict of plain values.  ``op`` names the operator; lengths follow from the case alone (its
``mix`` seeds them), tensor values from the seed given to ``prepare``."""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 500000.0
BLOCK = 128  # key block of the per-block e4m3 scale factors


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one short conversation on a small model: nothing but latency
        dict(name="decode 1x1024 d64", op="decode", dtype="bf16", Hq=4, Hkv=1, d=64, page=64, seqs=1,
             lo=1024, hi=1024, tokens=1, factors=False, mix=1),
        # a few chats of ordinary length
        dict(name="decode 8 ragged to 4097", op="decode", dtype="bf16", Hq=32, Hkv=8, d=128, page=64, seqs=8,
             lo=31, hi=4097, tokens=1, factors=False, mix=2),
        # one 128K context, contiguous cache
        dict(name="decode 1x131072", op="decode", dtype="bf16", Hq=32, Hkv=8, d=128, page=0, seqs=1,
             lo=131072, hi=131072, tokens=1, factors=False, mix=3),
        # eight long documents, 4K to 64K, e4m3 cache of permuted pages
        dict(name="decode 8 varlen e4m3", op="decode", dtype="fp8", Hq=32, Hkv=8, d=128, page=64, seqs=8,
             lo=4096, hi=65536, tokens=1, factors=False, mix=4),
        # a full batch of chats, small pages: the largest read
        dict(name="decode 128 ragged to 8191", op="decode", dtype="bf16", Hq=32, Hkv=8, d=128, page=16, seqs=128,
             lo=1, hi=8191, tokens=1, factors=False, mix=5),
        # four drafted tokens checked at once over a 256K context quantised per key block
        dict(name="decode 4 drafts 256K e4m3", op="decode", dtype="fp8", Hq=64, Hkv=8, d=128, page=64, seqs=1,
             lo=262144, hi=262144, tokens=4, factors=True, mix=6),
        # the new rows of one decode step
        dict(name="append 64x1", op="append", dtype="bf16", Hq=32, Hkv=8, d=128, page=64, seqs=64, tokens=1,
             prefix=65536, rot=128, interleaved=False, norm=True, pad=0, mix=7),
        # a prefill chunk deep in a 256K context, written to an e4m3 cache
        dict(name="append 32768 e4m3", op="append", dtype="fp8", Hq=64, Hkv=8, d=128, page=64, seqs=1, tokens=32768,
             prefix=229376, rot=128, interleaved=False, norm=True, pad=0, mix=8),
        # odd chunk lengths, half of the head rotated in adjacent pairs, contiguous cache, padded batch
        dict(name="append ragged half interleaved", op="append", dtype="bf16", Hq=8, Hkv=2, d=64, page=0, seqs=7, tokens=617,
             prefix=1000, rot=32, interleaved=True, norm=True, pad=13, mix=9),
        # the map of one decode step
        dict(name="map 64x1", op="map", page=64, seqs=64, new_lo=1, new_hi=1, prefix=65536, pad=0, mix=10),
        # a thousand requests with short prompts and decode rows mixed, small pages, padded batch
        dict(name="map 1000 mixed", op="map", page=16, seqs=1000, new_lo=0, new_hi=511, prefix=2047, pad=101, mix=11),
        # eight long prompts at once
        dict(name="map 8x32768", op="map", page=64, seqs=8, new_lo=32768, new_hi=32768, prefix=0, pad=0, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    op = rng.choice(["decode", "decode", "append", "map"])
    if op == "map":
        seqs = _log(rng, 1, 1000)
        hi = _log(rng, 1, max(1, 262144 // seqs))
        return dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), seqs=seqs, new_lo=rng.choice([0, 1]), new_hi=hi,
                    prefix=rng.choice([0, _log(rng, 1, 65536)]), pad=rng.choice([0, _log(rng, 1, 500)]), mix=mix)
    fp8 = rng.random() < 0.5
    Hq, Hkv, d = rng.choice([(32, 8, 128), (64, 8, 128), (16, 16, 128), (16, 8, 128)] + ([] if fp8 else [(4, 1, 64), (8, 2, 64)]))
    page = rng.choice([0, 16, 64, 128, 256])
    if op == "append":
        total = _log(rng, 1, 16384)
        seqs = _log(rng, 1, min(total, 256))
        return dict(op=op, dtype="fp8" if fp8 else "bf16", Hq=Hq, Hkv=Hkv, d=d, page=page, seqs=seqs, tokens=max(1, total // seqs),
                    prefix=rng.choice([0, _log(rng, 1, 229376)]), rot=rng.choice([d, d, d // 2, 0]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.8, pad=rng.choice([0, rng.randrange(1, 40)]), mix=mix)
    total = _log(rng, 200, 500000)
    seqs = _log(rng, 1, min(total, 128))
    hi = max(8, total // seqs)
    return dict(op=op, dtype="fp8" if fp8 else "bf16", Hq=Hq, Hkv=Hkv, d=d, page=page, seqs=seqs, lo=rng.choice([8, max(8, hi // 2), hi]), hi=hi,
                tokens=rng.choice([1, 1, 1, 2, 3, 5]), factors=fp8 and rng.random() < 0.5, mix=mix)


# ------------------------------------------------------ lengths of a case ---

def _decode_lens(c):
    r = random.Random(c["mix"])
    lk = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    lq = [1 if c["tokens"] == 1 else r.randint(0, min(k, c["tokens"])) for k in lk]  # drafts differ, and some rest this step
    at = r.randrange(len(lk))
    lk[at], lq[at] = c["hi"], c["tokens"]
    return lq, lk


def _append_lens(c):
    r = random.Random(c["mix"])
    if c["seqs"] == 1:
        return [c["tokens"]], [c["prefix"]]
    new = [c["tokens"] if c["tokens"] == 1 else r.randint(1, c["tokens"]) for _ in range(c["seqs"])]
    return new, [r.randint(0, c["prefix"]) for _ in new]


def _map_lens(c):
    r = random.Random(c["mix"])
    new = [r.randint(c["new_lo"], max(c["new_lo"], c["new_hi"])) for _ in range(c["seqs"])]
    return new, [r.randint(c["prefix"] // 2, c["prefix"]) for _ in new]


def _pages(lens, page, rs):
    """A page table of permuted physical pages for these lengths, unused entries -1, and its page count."""
    need = [-(-n // page) for n in lens]
    perm = rs.permutation(sum(need) + 2).astype(np.int32)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- prepare ---

def _quantised(shape, scale, g):
    """e4m3 rows [n, heads, d] of normal values, x = e4m3 * scale[head], made in pieces."""
    x = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for a in range(0, shape[0], 65536):
        n = min(65536, shape[0] - a)
        r = torch.randn((n,) + tuple(shape[1:]), generator=g, device="cuda")
        x[a:a + n] = (r / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + 13)
    rs = np.random.RandomState(seed % (1 << 31))
    return {"decode": _prepare_decode, "append": _prepare_append, "map": _prepare_map}[case["op"]](case, g, rs)


def _prepare_decode(c, g, rs):
    lq, lk = _decode_lens(c)
    Hq, Hkv, d, page, fp8 = c["Hq"], c["Hkv"], c["d"], c["page"], c["dtype"] == "fp8"
    s = dict(case=c, cu=_cu(lq), lk=_i32(lk), total_q=sum(lq), max_q=max(lq), max_k=max(lk), cu_k=None, table=None)
    if page:
        table, pages = _pages(lk, page, rs)
        s["table"], rows = _i32(table), pages * page
    else:
        s["cu_k"], rows = _cu(lk), sum(lk)
    if fp8:
        for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv)):  # scales that put a normal value's largest near the type's
            s[n + "_scale"] = 0.01 * (1 + 0.05 * torch.rand(h, generator=g, device="cuda"))
        s["q"] = _quantised((s["total_q"], Hq, d), s["q_scale"] * 0.5, g)  # queries of twice the keys' size
        s["k"], s["v"] = (_quantised((rows, Hkv, d), s[n + "_scale"], g) for n in "kv")
    else:
        s["q"] = (2 * torch.randn((s["total_q"], Hq, d), generator=g, device="cuda")).bfloat16()
        s["k"], s["v"] = (torch.randn((rows, Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    if page:
        s["k"], s["v"] = (s[n].view(-1, page, Hkv, d) for n in "kv")
    if c["factors"]:
        for n in "kv":  # per key block, in (0, 1]
            s[n + "_factor"] = 1 - 0.75 * torch.rand((c["seqs"], -(-s["max_k"] // BLOCK), Hkv), generator=g, device="cuda")
    return s


def _prepare_append(c, g, rs):
    new, prefix = _append_lens(c)
    Hq, Hkv, d, page, fp8 = c["Hq"], c["Hkv"], c["d"], c["page"], c["dtype"] == "fp8"
    live, total = sum(new), sum(new) + c["pad"]
    s = dict(case=c, live=live)
    s["qkv"] = torch.randn((total, (Hq + 2 * Hkv) * d), generator=g, device="cuda").bfloat16()  # the fused projection's rows
    s["w"] = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in "qk"] if c["norm"] else [None, None]
    s["inv_freq"] = (1.0 / THETA ** (torch.arange(0, c["rot"], 2, device="cuda").double() / max(1, c["rot"]))).float()
    pos = np.concatenate([p + np.arange(n) for p, n in zip(prefix, new)] + [np.zeros(c["pad"], int)])
    if page:
        # the pages that this chunk touches, at permuted places in the cache
        first = [p // page for p in prefix]
        count = [(p + n - 1) // page - f + 1 for p, n, f in zip(prefix, new, first)]
        perm, at, slots = rs.permutation(sum(count) + 1), 0, []
        for p, n, f, k in zip(prefix, new, first, count):
            t = p + np.arange(n)
            slots.append(perm[at + t // page - f] * page + t % page)
            at += k
        rows, slots = len(perm) * page, np.concatenate(slots)
    else:
        rows = live + 5
        slots = rs.permutation(rows)[:live]
    s["positions"], s["slots"] = _i32(pos), _i32(np.concatenate([slots, np.full(c["pad"], -1)]))
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    shape = (rows // page, page, Hkv, d) if page else (rows, Hkv, d)
    s["k_cache"], s["v_cache"] = (torch.zeros(shape, device="cuda").to(kind) for _ in "kv")
    s["q_out"] = torch.zeros((total, Hq, d), device="cuda").to(kind)
    if fp8:
        for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv)):
            s[n + "_scale"] = 0.012 * (1 + 0.05 * torch.rand(h, generator=g, device="cuda"))
    return s


def _prepare_map(c, g, rs):
    new, prefix = _map_lens(c)
    page = c["page"]
    old = [-(-p // page) for p in prefix]
    after = [-(-(p + n) // page) for p, n in zip(prefix, new)]
    pages = sum(after) + 7
    perm, table, at = rs.permutation(pages).astype(np.int32), np.full((len(new), max(1, max(after))), -1, np.int32), 0
    for b, n in enumerate(old):
        table[b, :n] = perm[at:at + n]
        at += n
    used = 3  # entries of the free list that earlier steps have taken
    free = np.concatenate([perm[:used], perm[at:]])
    return dict(case=c, total=sum(new) + c["pad"], pages=pages, table=_i32(table), new=_i32(new), prefix=_i32(prefix), free=_i32(free),
                head=_i32([used]), max_new=max(new), max_k=max(1, max(p + n for p, n in zip(prefix, new))))


# -------------------------------------------------------------------- run ---

def run(s):
    op = s["case"]["op"]
    if own:
        return {"decode": _own_decode, "append": _own_append, "map": _own_map}[op](s)
    return {"decode": _plain_decode, "append": _plain_append, "map": _plain_map}[op](s)


def _own_decode(s):
    from block_sparse_long_blockmean_b200 import fp2
    c = s["case"]
    if "plan" not in s:  # the handle that a serving loop keeps: parameters, workspace, output buffers
        s["plan"] = fp2.make_decode(
            s["q"], s["k"], s["v"], s["cu"], Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"], block=BLOCK,
            dtype=fp2.FP2_FP8_E4M3 if c["dtype"] == "fp8" else fp2.FP2_BF16, max_seqlen_q=s["max_q"], max_seqlen_k=s["max_k"],
            seqlens_k=s["lk"], cu_seqlens_k=s["cu_k"], page_table=s["table"], page_size=c["page"], q_scale=s.get("q_scale"),
            k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), k_block_factor=s.get("k_factor"), v_block_factor=s.get("v_factor"),
            with_lse=True)
    s["plan"].run()
    return {"out": s["plan"].out, "lse": s["plan"].lse}


def _own_append(s):
    from block_sparse_long_blockmean_b200 import fp2
    c = s["case"]
    if "plan" not in s:
        Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
        q, k, v = (x.view(-1, h, d) for x, h in zip(s["qkv"].split([Hq * d, Hkv * d, Hkv * d], dim=1), (Hq, Hkv, Hkv)))
        s["plan"] = fp2.make_append(
            q, k, v, s["k_cache"], s["v_cache"], s["positions"], s["slots"], dtype=fp2.FP2_FP8_E4M3 if c["dtype"] == "fp8" else fp2.FP2_BF16,
            inv_freq=s["inv_freq"], rotary_dim=c["rot"], interleaved=c["interleaved"], q_weight=s["w"][0], k_weight=s["w"][1], eps=EPS,
            q_scale=s.get("q_scale"), k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), q_out=s["q_out"])
    s["plan"].run()
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_map(s):
    from block_sparse_long_blockmean_b200 import fp2
    if "plan" not in s:
        s["plan"] = fp2.make_page_map(s["prefix"], s["new"], s["table"], s["free"], s["head"], page_size=s["case"]["page"],
                                      num_pages=s["pages"], total_q=s["total"], max_seqlen_q=s["max_new"], max_seqlen_k=s["max_k"])
    m = s["plan"]
    m.run()
    return {"cu_seqlens": m.cu_seqlens, "seqlens_k": m.seqlens_k, "positions": m.positions, "slot_map": m.slot_map, "page_table": m.page_table,
            "free_head": m.free_head_out}


def _rows(cache, at):
    """Rows `at` of a cache [.., Hkv, d], as 32-bit values."""
    flat = cache.reshape(-1, *cache.shape[-2:])
    if flat.dtype == torch.float8_e4m3fn:
        return flat.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return flat[at].float()


def _plain_decode(s):
    c, cu, lk = s["case"], s["cu"].long(), s["lk"].long()
    Hq, Hkv, d, page, T, L = c["Hq"], c["Hkv"], c["d"], c["page"], s["max_q"], s["max_k"]
    S, G, dev = c["seqs"], c["Hq"] // c["Hkv"], cu.device
    j, t = torch.arange(L, device=dev), torch.arange(T, device=dev)
    if page:
        at = s["table"].long().clamp(min=0)[:, j // page] * page + j % page
    else:
        at = (s["cu_k"][:-1].long()[:, None] + j).clamp(max=s["k"].shape[0] - 1)
    q, k, v = s["q"].float(), _rows(s["k"], at), _rows(s["v"], at)
    if c["dtype"] == "fp8":
        q, ks, vs = q * s["q_scale"][:, None], s["k_scale"].expand(S, L, Hkv), s["v_scale"].expand(S, L, Hkv)
        if c["factors"]:
            ks, vs = ks * s["k_factor"][:, j // BLOCK], vs * s["v_factor"][:, j // BLOCK]
        k, v = k * ks[..., None], v * vs[..., None]
    lq = cu[1:] - cu[:-1]
    q = q[(cu[:-1, None] + t).clamp(max=s["total_q"] - 1)].view(S, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * T, d)
    logits = (q @ k.permute(0, 2, 3, 1)).view(S, Hkv, G, T, L) * (1 / math.sqrt(d))
    seen = j <= ((lk - lq)[:, None] + t).clamp(max=L - 1)[:, :, None]                      # [S, T, L], key j of query t
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    m = logits.amax(-1, keepdim=True)
    p = (logits - m).exp()
    l = p.sum(-1, keepdim=True)
    o = (p.view(S, Hkv, G * T, L) @ v.permute(0, 2, 1, 3)).view(S, Hkv, G, T, d) / l
    i = torch.arange(s["total_q"], device=dev)
    b = torch.searchsorted(cu[1:], i, right=True)
    t = i - cu[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, t].reshape(-1, Hq, d).bfloat16(),
            "lse": (m + l.log())[..., 0].permute(0, 3, 1, 2)[b, t].reshape(-1, Hq)}


def _rotated(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), x[..., rot:]], -1)


def _stored(x, like, scale):
    if like.dtype == torch.float8_e4m3fn:
        return (x / scale[:, None]).clamp(-448, 448).to(like.dtype)
    return x.to(like.dtype)


def _put(cache, slots, rows):
    flat = cache.view(-1, *cache.shape[-2:])
    if flat.dtype == torch.float8_e4m3fn:
        flat, rows = flat.view(torch.uint8), rows.view(torch.uint8)
    flat[slots] = rows


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, d, rot, live = c["Hq"], c["Hkv"], c["d"], c["rot"], s["live"]
    q, k, v = (x.float().view(-1, h, d) for x, h in zip(s["qkv"].split([Hq * d, Hkv * d, Hkv * d], dim=1), (Hq, Hkv, Hkv)))
    if c["norm"]:
        q, k = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w for x, w in zip((q, k), s["w"]))
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = (_rotated(x, cos, sin, rot, c["interleaved"]) for x in (q, k))
    s["q_out"].copy_(_stored(q, s["q_out"], s.get("q_scale")))
    slots = s["slots"][:live].long()
    _put(s["k_cache"], slots, _stored(k[:live], s["k_cache"], s.get("k_scale")))
    _put(s["v_cache"], slots, _stored(v[:live], s["v_cache"], s.get("v_scale")))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_map(s):
    page, prefix, new, table, free = s["case"]["page"], s["prefix"], s["new"], s["table"], s["free"]
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    old = (prefix + page - 1) // page
    need = (prefix + new + page - 1) // page - old
    taken = need.cumsum(0)
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    at = s["head"] + (taken - need)[:, None] + col - old[:, None]
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    i = torch.arange(s["total"], device=table.device)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=new.numel() - 1)
    pos = prefix[b] + i - cu[b]
    live = i < cu[-1]
    pos = torch.where(live, pos, 0)
    slot = torch.where(live, table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page, -1)
    return {"cu_seqlens": cu.int(), "seqlens_k": prefix + new, "positions": pos.int(), "slot_map": slot.int(), "page_table": table,
            "free_head": (s["head"] + taken[-1]).int()}


# ------------------------------------------------------------------- work ---

def work(case):
    c = case
    if c["op"] == "map":
        new, prefix = _map_lens(c)
        fresh = sum(-(-(p + n) // c["page"]) - -(-p // c["page"]) for p, n in zip(prefix, new))
        total = sum(new) + c["pad"]
        return {"bytes": 16 * c["seqs"] + 8 * fresh + 8 * total, "flops": 4 * total}
    e = 1 if c["dtype"] == "fp8" else 2
    if c["op"] == "append":
        total, width = sum(_append_lens(c)[0]) + c["pad"], (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        kept = total * c["Hq"] * c["d"] + (total - c["pad"]) * 2 * c["Hkv"] * c["d"]
        return {"bytes": 2 * total * width + e * kept + 8 * total, "flops": 9 * total * (c["Hq"] + c["Hkv"]) * c["d"]}
    lq, lk = _decode_lens(c)
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(lq, lk))
    lk = [k for q, k in zip(lq, lk) if q]
    read = 2 * sum(lk) * c["Hkv"] * c["d"] * e
    if c["factors"]:
        read += 8 * sum(-(-k // BLOCK) for k in lk) * c["Hkv"]
    if c["page"]:
        read += 4 * sum(-(-k // c["page"]) for k in lk)
    return {"bytes": read + sum(lq) * c["Hq"] * (c["d"] * (e + 2) + 4), "flops": 4 * pairs * c["Hq"] * c["d"]}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "map": _exact_map}[case["op"]](case, s)


def _exact_decode(c, s):
    """Sequence by sequence and head by head, from the definition."""
    cu, lk, G, page = s["cu"].tolist(), s["lk"].tolist(), c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros((s["total_q"], c["Hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total_q"], c["Hq"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lk):
        if page:
            pages = s["table"][b, :-(-n // page)].long()
            K, V = (x.view(torch.uint8)[pages].view(x.dtype).reshape(-1, c["Hkv"], c["d"])[:n] for x in (s["k"], s["v"]))
        else:
            a = int(s["cu_k"][b])
            K, V = s["k"][a:a + n], s["v"][a:a + n]
        rows = slice(cu[b], cu[b + 1])
        first = n - (cu[b + 1] - cu[b])  # keys before the first new token
        visible = torch.ones((cu[b + 1] - cu[b], n), dtype=torch.bool, device="cuda").tril(first)
        for h in range(c["Hkv"]):
            k, v = K[:, h].double(), V[:, h].double()
            if c["dtype"] == "fp8":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
                if c["factors"]:
                    k *= s["k_factor"][b, :, h].double().repeat_interleave(BLOCK)[:n, None]
                    v *= s["v_factor"][b, :, h].double().repeat_interleave(BLOCK)[:n, None]
            for hq in range(h * G, (h + 1) * G):
                q = s["q"][rows, hq].double() * (s["q_scale"][hq].double() if c["dtype"] == "fp8" else 1.0)
                z = (q @ k.T) / math.sqrt(c["d"])
                z[~visible] = -math.inf
                out[rows, hq] = torch.softmax(z, -1) @ v
                lse[rows, hq] = torch.logsumexp(z, -1)
    return {"out": out, "lse": lse}


def _exact_append(c, s):
    """Rotation as a product of complex numbers, in 64 bits; e4m3 outputs in units of their scales."""
    Hq, Hkv, d, rot = c["Hq"], c["Hkv"], c["d"], c["rot"]
    x = s["qkv"].double().view(-1, Hq + 2 * Hkv, d)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    turn = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]

    def placed(y, w):
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        y = y.clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y

    def unit(y, name):
        return (y / s[name + "_scale"].double()[:, None]).clamp(-448, 448) if c["dtype"] == "fp8" else y

    got = {"q": unit(placed(q, s["w"][0]), "q")}
    at = s["slots"][:s["live"]].long()
    for name, rows in (("k", placed(k, s["w"][1])), ("v", v)):
        cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda")
        cache.view(-1, Hkv, d)[at] = unit(rows, name)[:s["live"]]
        got[name + "_cache"] = cache
    return got


def _exact_map(c, s):
    """Request by request on the host, as an allocator would."""
    page, new, prefix = c["page"], s["new"].tolist(), s["prefix"].tolist()
    table, free, head = s["table"].cpu().numpy().copy(), s["free"].tolist(), int(s["head"])
    cu, pos, slots = [0], [], []
    for b, (n, p) in enumerate(zip(new, prefix)):
        for k in range(-(-p // page), -(-(p + n) // page)):
            table[b, k] = free[head]
            head += 1
        t = np.arange(p, p + n)
        pos.append(t)
        slots.append(table[b, t // page] * page + t % page)
        cu.append(cu[-1] + n)
    pos, slots = (np.concatenate(x + [np.full(c["pad"], e)]) for x, e in ((pos, 0), (slots, -1)))
    return {"cu_seqlens": _i32(cu), "seqlens_k": s["prefix"] + s["new"], "positions": _i32(pos), "slot_map": _i32(slots), "page_table": _i32(table),
            "free_head": _i32([head])}
