"""Measured cases of the operators between a fused QKV projection and a verified draft tree.

Five operators, in the order a program calls them:

* qk_norm_rope:  per-head RMS norms of q and k and the position rotation, one pass
* append_rope:   q, k normalised and rotated, k and v Hadamard-rotated, quantised to 4 bits and
                 placed in pages (the rows written are read back as values, so that they can be compared)
* prompt:        causal attention of packed prompts over their own BF16 rows
* tree:          attention of drafted token trees over the paged 4-bit cache
* move:          the entries of an accepted branch moved to consecutive positions

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits (angles in
64); where it is true, through the library's entry points.  ``exact`` computes what they are defined to
be in 64 bits.

A page of the cache holds, for each KV head, P positions: P K entries of d/2 bytes, P/2 V entries (one
for two positions) of d bytes, and P pairs of BF16 scales (K, V).  Values are sign and magnitude (0..7),
four to a 16-bit word with channels 32 j + g + {0, 8, 16, 24}: magnitudes at bits 0, 3, 8, 11 and signs
at bits 15, 14, 7, 6.
"""
import math
import random

import torch

own = False

MAG = (0, 3, 8, 11)
SGN = (15, 14, 7, 6)
BASE, EPS = 500000.0, 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # q and k of one token for each of 32 requests, 8B-shaped layer with per-head norms: latency
        {"name": "qk_step_b32", "op": "qk", "n_q": 32, "n_kv": 8, "d": 128, "batch": 32, "new": 1, "ctx": 4096, "norm": True, "seed": 1},
        # packed prompts of up to 2048 tokens after their projection
        {"name": "qk_prompts_32k", "op": "qk", "n_q": 32, "n_kv": 8, "d": 128, "batch": 16, "new": 2048, "ctx": 0, "norm": True, "seed": 2},
        # the drafted tokens of 8 requests, 70B-shaped layer without norms, far positions
        {"name": "append_drafts_70b", "op": "append", "n_q": 64, "n_kv": 8, "d": 128, "had": 128, "batch": 8, "new": 24, "ctx": 100000,
         "page": 64, "norm": False, "seed": 3},
        # chunks of prompts placed with their queries prepared
        {"name": "append_chunks_16k", "op": "append", "n_q": 32, "n_kv": 8, "d": 128, "had": 128, "batch": 8, "new": 2048, "ctx": 2000,
         "page": 32, "norm": True, "seed": 4},
        # one short prompt: latency
        {"name": "prompt_8b_100", "op": "prompt", "n_q": 32, "n_kv": 8, "d": 128, "batch": 1, "new": 100, "ragged": False, "seed": 5},
        # prompts of a small model (head_dim 64) of odd, unequal lengths
        {"name": "prompt_d64_ragged", "op": "prompt", "n_q": 8, "n_kv": 2, "d": 64, "batch": 9, "new": 1111, "ragged": True, "seed": 6},
        # a batch of prompts as a server packs them
        {"name": "prompt_8b_8x2048", "op": "prompt", "n_q": 32, "n_kv": 8, "d": 128, "batch": 8, "new": 2048, "ragged": True, "seed": 7},
        # one long document, 8B shape
        {"name": "prompt_8b_8192", "op": "prompt", "n_q": 32, "n_kv": 8, "d": 128, "batch": 1, "new": 8192, "ragged": False, "seed": 8},
        # small trees of a serving batch: 7 drafted tokens for each of 32 requests of up to 4096
        {"name": "tree_8b_b32_7", "op": "tree", "n_q": 32, "n_kv": 8, "d": 128, "had": 128, "batch": 32, "nodes": 7, "kv": 4096, "page": 64,
         "ragged": True, "seed": 9},
        # a wide tree of one request over a long context, 70B shape
        {"name": "tree_70b_b1_64", "op": "tree", "n_q": 64, "n_kv": 8, "d": 128, "had": 128, "batch": 1, "nodes": 64, "kv": 32768, "page": 64,
         "ragged": False, "seed": 10},
        # accepted branches of 32 requests
        {"name": "move_b32", "op": "move", "n_kv": 8, "d": 128, "batch": 32, "nodes": 24, "keep": 5, "page": 64, "seed": 11},
        # long accepted branches of a large batch, small pages
        {"name": "move_b256", "op": "move", "n_kv": 8, "d": 128, "batch": 256, "nodes": 128, "keep": 32, "page": 16, "seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("qk", "append", "prompt", "prompt", "tree", "tree", "move"))
    seed, page = rng.randrange(1 << 20), rng.choice((16, 32, 64, 128))
    n_kv, g, d = rng.choice(((8, 4, 128), (8, 8, 128), (2, 4, 64), (4, 1, 128), (6, 7, 64), (4, 3, 128)))
    had = rng.choice((d, d, d, 32, 1))
    if op in ("qk", "append"):
        batch = _log(rng, 1, 64)
        c = {"op": op, "n_q": n_kv * g, "n_kv": n_kv, "d": d, "batch": batch, "new": rng.choice((1, _log(rng, 1, 12288 // batch))),
             "ctx": _log(rng, 1, 1000000), "norm": rng.random() < 0.5, "seed": seed}
        return c if op == "qk" else c | {"had": had, "page": page, "ctx": _log(rng, 1, 4096)}
    if op == "prompt":
        batch = _log(rng, 1, 16)
        return {"op": op, "n_q": n_kv * g, "n_kv": n_kv, "d": d, "batch": batch, "new": _log(rng, 1, 4096 // math.isqrt(batch)),
                "ragged": rng.random() < 0.7, "seed": seed}
    if op == "tree":
        batch = _log(rng, 1, 32)
        nodes = _log(rng, 1, 128 if batch <= 8 else 32)
        return {"op": op, "n_q": n_kv * g, "n_kv": n_kv, "d": d, "had": had, "batch": batch, "nodes": nodes,
                "kv": nodes + _log(rng, 1, min(32000, 65536 // batch)), "page": page, "ragged": rng.random() < 0.7, "seed": seed}
    nodes = _log(rng, 1, 128)
    return {"op": op, "n_kv": n_kv, "d": d, "batch": _log(rng, 1, 256), "nodes": nodes, "keep": rng.randint(1, nodes), "page": page, "seed": seed}


def lengths(case):
    """(tokens to add, tokens afterwards) of each request: the longest first, then any shorter ones."""
    r, b, op = random.Random(case["seed"]), case["batch"], case["op"]
    if op == "move":
        new = [case["nodes"]] * b
        return new, [n + r.randint(0, 100) for n in new]
    if op == "tree":
        new = [case["nodes"]] + [r.randint(1, case["nodes"]) if case["ragged"] else case["nodes"] for _ in range(b - 1)]
        kv = [case["kv"]] + [r.randint(1, case["kv"]) if case["ragged"] else case["kv"] for _ in range(b - 1)]
        return new, [max(n, k) for n, k in zip(new, kv)]
    ragged = case.get("ragged", True)
    new = [case["new"]] + [r.randint(1, case["new"]) if ragged else case["new"] for _ in range(b - 1)]
    return new, [n + (r.randint(0, case["ctx"]) if op != "prompt" else 0) for n in new]


def trees(case):
    """Parent of each drafted token, request by request (-1: the last token of the history)."""
    r = random.Random(case["seed"] + 1)
    return [[r.choice((-1, i - 1, r.randint(-1, i - 1), i - 1)) if i else -1 for i in range(n)] for n in lengths(case)[0]]


def branches(case):
    """What is kept of each request's drafted tokens: ascending places, at most `keep` of them."""
    r = random.Random(case["seed"] + 2)
    return [sorted(r.sample(range(case["nodes"]), r.randint(1, case["keep"]))) for _ in range(case["batch"])]


def work(case):
    op, (new, kv) = case["op"], lengths(case)
    total, h, d = sum(new), case["n_kv"], case["d"]
    if op == "move":
        moved = sum(sum(i != j for j, i in enumerate(keep)) for keep in branches(case))
        # slots read, entries read and written
        return {"bytes": 8 * case["batch"] * case["keep"] + 2 * moved * h * (d + 4), "flops": float(moved)}
    n_q = case["n_q"]
    if op == "qk":
        return {"bytes": total * (4 + 4 * (n_q + h) * d), "flops": 10.0 * total * (n_q + h) * d}
    if op == "append":
        # BF16 rows and slots read, queries and entries written, entries read again, BF16 values written
        return {"bytes": total * (8 + 4 * n_q * d + h * (4 * d + 2 * (d + 4) + 4 * d)),
                "flops": total * (10.0 * (n_q + h) * d + 2 * h * d * (2 * math.log2(d) + 4))}
    if op == "prompt":
        return {"bytes": 4 * total * (n_q + h) * d, "flops": 4.0 * d * n_q * sum(n * (n + 1) // 2 for n in new)}
    pairs = 0
    for n, k, parent in zip(new, kv, trees(case)):
        depth = []
        for up in parent:
            depth.append(1 + (depth[up] if up >= 0 else 0))
        pairs += n * (k - n) + sum(depth)
    return {"bytes": sum(kv) * h * (d + 4) + 4 * total * n_q * d + 4 * total * -(-case["nodes"] // 32) + 4 * sum(-(-k // case["page"]) for k in kv),
            "flops": 4.0 * d * n_q * pairs}


# ------------------------------------------------------------------ inputs
def _gen(case, seed):
    return torch.Generator("cuda").manual_seed((case["seed"] * 1000003 + seed) % (1 << 62))


def _halfwords(mag, neg):
    """[..., d] magnitudes and signs (int32) -> int16 [..., j, g]: channel 32 j + 8 e + g is value e."""
    m, s = (t.unflatten(-1, (-1, 4, 8)) for t in (mag, neg))
    w = (m[..., 0, :] << MAG[0]) | (m[..., 1, :] << MAG[1]) | (m[..., 2, :] << MAG[2]) | (m[..., 3, :] << MAG[3])
    w = w | (s[..., 0, :] << SGN[0]) | (s[..., 1, :] << SGN[1]) | (s[..., 2, :] << SGN[2]) | (s[..., 3, :] << SGN[3])
    return (w - ((w & 0x8000) << 1)).to(torch.int16)


def _chunk_of(pair, d):
    """[n] pair numbers -> [n, 8]: where chunk g of a V entry is stored."""
    g = torch.arange(8, device=pair.device)
    return g[None, :] ^ (2 * (pair & 3) if d == 128 else 4 * ((pair >> 1) & 1))[:, None]


def _pool(n_pages, n_kv, page, d, gen):
    """Pages of random entries, distributed as the quantiser leaves rotated keys and values: about normal, largest 7."""
    out = torch.empty((n_pages, n_kv, page * (d + 4)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (n_kv * page * d))
    at = _chunk_of(torch.arange(page // 2, device="cuda"), d)
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        words = []
        for _ in range(2):
            c = (torch.randn((b - a, n_kv, page, d), device="cuda", generator=gen) * 2.6).round_().clamp_(-7, 7).to(torch.int32)
            words.append(_halfwords(c.abs(), (c < 0).to(torch.int32)))
        k, v = words  # [n, h, P, j, g]
        k = k.unflatten(-1, (4, 2)).permute(0, 1, 2, 4, 3, 5).reshape(b - a, n_kv, -1)
        v = v.unflatten(2, (-1, 2)).permute(0, 1, 2, 5, 4, 3)  # [n, h, pair, g, j, half]
        v = torch.empty_like(v, memory_format=torch.contiguous_format).scatter_(3, at[None, None, :, :, None, None].expand_as(v), v)
        s = torch.exp(0.3 * torch.randn((b - a, n_kv, page, 2), device="cuda", generator=gen) - 1).to(torch.bfloat16)
        out[a:b] = torch.cat((k, v.reshape(b - a, n_kv, -1), s.view(torch.int16).reshape(b - a, n_kv, -1)), -1).view(torch.uint8)
    return out


def _tables(case, kv, gen):
    """Block tables of requests holding kv tokens, their pages scattered over the pool; -1 behind the last one."""
    p, need = case["page"], [-(-k // case["page"]) for k in kv]
    n_pages = sum(need) + 3
    ids = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    at = torch.tensor([0] + need).cumsum(0)
    col = torch.arange(max(need) + 1, device="cuda")[None, :]
    idx = at[:-1, None].cuda() + col
    table = torch.where(col < torch.tensor(need).cuda()[:, None], ids[idx.clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return n_pages, table.contiguous()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _prefix(v):
    return _ints([0] + torch.tensor(v).cumsum(0).tolist())


def _projected(total, heads, d, gen):
    """BF16 rows of a fused projection: normal values and the few outlier channels of real keys."""
    x = torch.randn((total, heads, d), device="cuda", generator=gen)
    hot = torch.randint(0, d, (1, heads, 2), device="cuda", generator=gen).expand(total, -1, -1)
    return x.scatter(2, hot, x.gather(2, hot) * 8).to(torch.bfloat16)


def prepare(case, seed):
    gen, op = _gen(case, seed), case["op"]
    new, kv = lengths(case)
    h, d, total, b = case["n_kv"], case["d"], sum(new), len(new)
    s = {"case": case, "total": total, "B": b, "cu": _prefix(new)}
    empty = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if op != "move":
        n_q = case["n_q"]
    if op in ("qk", "append", "prompt"):
        buf = _projected(total, n_q + 2 * h, d, gen)
        s["q"], s["k"], s["v"] = buf[:, :n_q], buf[:, n_q:n_q + h], buf[:, n_q + h:]
    if op in ("qk", "append"):
        req = torch.repeat_interleave(torch.arange(b), torch.tensor(new))
        pos = torch.arange(total) - s["cu"].cpu()[req] + torch.tensor([k - n for n, k in zip(new, kv)])[req]
        s["pos"] = pos.to(torch.int32).cuda()
        gain = lambda: 1 + 0.3 * torch.randn((d,), device="cuda", generator=gen) if case["norm"] else None  # noqa: E731
        s["gq"], s["gk"] = gain(), gain()
        s["q_out"] = empty(total, n_q, d)
    if op == "qk":
        s["k_out"] = empty(total, h, d)
    if op == "prompt":
        s["max"], s["o"] = max(new), empty(total, n_q, d)
    if op == "append":  # pages for the new tokens alone
        s["n_pages"], table = _tables(case, new, gen)
        p, i = case["page"], (torch.arange(total) - s["cu"].cpu()[req]).cuda()
        s["slots"] = (table[req.cuda(), i // p] * p + (i % p).to(torch.int32)).contiguous()
        s["pool"] = torch.zeros((s["n_pages"], h, p * (d + 4)), dtype=torch.uint8, device="cuda")
        s["k_out"], s["v_out"] = empty(total, h, d), empty(total, h, d)
    if op in ("tree", "move"):
        s["n_pages"], s["table"] = _tables(case, kv, gen)
        s["pool"] = _pool(s["n_pages"], h, case["page"], d, gen)
    if op == "tree":
        s["kv_len"], s["max_q"], s["max_kv"], words = _ints(kv), max(new), max(kv), -(-case["nodes"] // 32)
        rows = []
        for parent in trees(case):
            first = len(rows)
            for i, up in enumerate(parent):
                rows.append((rows[first + up] if up >= 0 else 0) | 1 << i)
        cut = lambda x: x - (1 << 32) if x >> 31 else x  # noqa: E731
        s["mask"] = _ints([[cut(x >> 32 * w & 0xFFFFFFFF) for w in range(words)] for x in rows])
        s["q"] = torch.randn((total, n_q, d), device="cuda", generator=gen).to(torch.bfloat16)
        s["o"] = empty(total, n_q, d)
    if op == "move":
        p = case["page"]
        src, dst = (torch.full((b, case["keep"]), -1, dtype=torch.int64) for _ in range(2))
        table = s["table"].cpu()
        for r, keep in enumerate(branches(case)):
            for out, places in ((src, torch.tensor(keep)), (dst, torch.arange(len(keep)))):
                at = places + kv[r] - new[r]
                out[r, :len(keep)] = table[r, at // p] * p + at % p
        s["src"], s["dst"] = src.to(torch.int32).cuda(), dst.to(torch.int32).cuda()
    if own:
        import int4_weight_kv_gb300 as ft

        n_q = case.get("n_q") or h
        s["cfg"] = ft.make_cfg(128 * n_q, n_q, h, d, 128, had_block=case.get("had", 0), rms_eps=EPS, rope_base=BASE)
        if op == "tree":
            size = ft.ft_attn_tree_workspace_bytes(s["cfg"], b, total, s["max_q"])
            s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms
def _butterfly(x, block):
    """x times the normalised Sylvester matrix of order `block`, in 32 bits, strides 1, 2, 4, ... in this order."""
    n, s = x.shape, 1
    while s < block:
        y = x.reshape(-1, 2, s)
        x = torch.stack((y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]), 1)
        s *= 2
    return x.reshape(n) * (float(block) ** -0.5)


def _values(words, scale):
    """int16 [..., j, g] and scales [...] -> values [..., d]."""
    w = words.to(torch.int32)
    e = [((w >> MAG[i]) & 7) * (1 - 2 * ((w >> SGN[i]) & 1)) for i in range(4)]
    return torch.stack(e, -2).flatten(-3).to(torch.float32) * scale[..., None]


def _decode(blocks, page, d):
    """Head blocks uint8 [..., page (d + 4)] -> K and V values [..., page, d]."""
    w = blocks.view(torch.int16)
    n = page * d // 4
    k = w[..., :n].unflatten(-1, (page, 4, d // 32, 2)).transpose(-3, -2).flatten(-2)  # [.., P, j, g]
    v = w[..., n:2 * n].unflatten(-1, (page // 2, 8, d // 32, 2))
    at = _chunk_of(torch.arange(page // 2, device=w.device), d)
    v = torch.gather(v, -3, at[:, :, None, None].expand(v.shape)).permute(*range(v.dim() - 4), -4, -1, -2, -3).flatten(-4, -3)
    s = w[..., 2 * n:].contiguous().view(torch.bfloat16).unflatten(-1, (page, 2)).float()
    return _values(k, s[..., 0]), _values(v, s[..., 1])


def _quantise(x, had):
    """FP32 rows -> int16 words [..., j, g] and BF16 scales of the rotated rows."""
    r = _butterfly(x, had)
    amax = r.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).to(torch.bfloat16)
    f = s.float()[..., None]
    c = torch.where(f == 0, torch.zeros_like(r), r / torch.where(f == 0, torch.ones_like(f), f))
    c = c.round().clamp(-7, 7).to(torch.int32)
    return _halfwords(c.abs(), (c < 0).to(torch.int32)), s


def _places(slot, page, n_kv, d):
    """Where in the pool's 16-bit words an entry's K words, V words [T, h, j, g] and scales [T, h] are."""
    inside = slot % page
    block = ((slot // page)[:, None] * n_kv + torch.arange(n_kv, device="cuda")) * (page * (d + 4) // 2)  # [T, h]
    j, g = torch.arange(d // 32, device="cuda")[:, None], torch.arange(8, device="cuda")[None, :]
    k_in = (inside * (d // 4))[:, None, None] + (g >> 1) * (d // 16) + 2 * j + (g & 1)
    chunk = _chunk_of(inside >> 1, d)
    v_in = page * d // 4 + ((inside >> 1) * (d // 2))[:, None, None] + chunk[:, None, :] * (d // 16) + 2 * j + (inside & 1)[:, None, None]
    s_in = page * d // 2 + 2 * inside
    return block[:, :, None, None] + k_in[:, None], block[:, :, None, None] + v_in[:, None], block + s_in[:, None]


def _turned(x, gain, pos):
    """Rows [T, heads, d] normalised per head and rotated to their positions, in 32 bits (angles in 64)."""
    x, d = x.float(), x.shape[-1]
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    a = pos.double()[:, None] * BASE ** (torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / -d)
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    u, w = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((u * c - w * s, w * c + u * s), -1)


def _plain_qk(s):
    return {"q": _turned(s["q"], s["gq"], s["pos"]).to(torch.bfloat16), "k": _turned(s["k"], s["gk"], s["pos"]).to(torch.bfloat16)}


def _plain_append(s):
    c = s["case"]
    flat = s["pool"].view(torch.int16).view(-1)
    k_at, v_at, s_at = _places(s["slots"].long(), c["page"], c["n_kv"], c["d"])
    kw, ks = _quantise(_turned(s["k"], s["gk"], s["pos"]), c["had"])
    vw, vs = _quantise(s["v"].float(), c["had"])
    flat[k_at], flat[v_at] = kw, vw
    flat[s_at], flat[s_at + 1] = ks.view(torch.int16), vs.view(torch.int16)
    back = lambda at, e: _butterfly(_values(flat[at], flat[s_at + e].view(torch.bfloat16).float()), c["had"]).to(torch.bfloat16)  # noqa: E731
    return {"q": _turned(s["q"], s["gq"], s["pos"]).to(torch.bfloat16), "k": back(k_at, 0), "v": back(v_at, 1)}


def _plain_move(s):
    c, flat = s["case"], s["pool"].view(torch.int16).view(-1)
    src, dst = s["src"].flatten().long(), s["dst"].flatten().long()
    there = (src >= 0) & (dst >= 0)
    src, dst = src[there], dst[there]
    for a, b in zip(_places(src, c["page"], c["n_kv"], c["d"]), _places(dst, c["page"], c["n_kv"], c["d"])):
        flat[b] = flat[a]
        if a.dim() == 2:
            flat[b + 1] = flat[a + 1]
    return s["pool"]


def _soft(q, k, v, seen, scale):
    """q [..., g, n, d], k and v [..., L, d], seen [..., n, L] -> [..., g, n, d]; a row that sees nothing: zeros."""
    sc = (q.flatten(-3, -2) @ k.transpose(-1, -2)).unflatten(-2, q.shape[-3:-1]) * scale
    sc = sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    e = sc.sub_(m).exp_()
    return (e.flatten(-3, -2) @ v).unflatten(-2, q.shape[-3:-1]) / e.sum(-1, keepdim=True)


def _padded(s, x, n):
    """Packed rows [T, heads, d] -> [B, n, heads, d], each request's rows from its first on."""
    cu = s["cu"].long()
    return x[(cu[:-1, None] + torch.arange(n, device="cuda")).clamp(max=s["total"] - 1)]


def _packed(s, o):
    """[B, n, heads, d] -> [T, heads, d]."""
    cu = s["cu"].long()
    req = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), cu[1:] - cu[:-1], output_size=s["total"])
    return o[req, torch.arange(s["total"], device="cuda") - cu[req]]


def _plain_prompt(s):
    c, n = s["case"], s["max"]
    h = c["n_kv"]
    q, k, v = (_padded(s, s[x].float(), n).transpose(1, 2) for x in ("q", "k", "v"))  # [B, heads, n, d]
    i = torch.arange(n, device="cuda")
    o = _soft(q.unflatten(1, (h, -1)), k, v, i[None, :] <= i[:, None], c["d"] ** -0.5)  # [B, h, g, n, d]
    return _packed(s, o.flatten(1, 2).transpose(1, 2)).to(torch.bfloat16)


def _plain_tree(s):
    c = s["case"]
    d, h, p, n = c["d"], c["n_kv"], c["page"], s["max_q"]
    pages = -(-s["max_kv"] // p)
    k, v = _decode(s["pool"][s["table"][:, :pages].clamp(min=0).long()], p, d)  # [B, pages, h, P, d]
    k, v = (t.transpose(1, 2).flatten(2, 3) for t in (k, v))  # [B, h, L, d]
    q = _padded(s, _butterfly(s["q"].float(), c["had"]), n).transpose(1, 2).unflatten(1, (h, -1))  # [B, h, g, n, d]
    cu = s["cu"].long()
    fresh = torch.arange(pages * p, device="cuda") - (s["kv_len"] - (cu[1:] - cu[:-1]))[:, None]  # [B, L]: which new token
    bits = _padded(s, s["mask"], n)  # [B, n, words]
    word = (fresh.clamp(0, n - 1) // 32)[:, None, :].expand(-1, n, -1)
    seen = (torch.gather(bits, 2, word) >> (fresh.clamp(min=0) % 32)[:, None, :]) & 1
    seen = (fresh < 0)[:, None] | ((seen == 1) & (fresh < (cu[1:] - cu[:-1])[:, None])[:, None])
    o = _soft(q, k, v, seen[:, None, None], d ** -0.5)
    o = _butterfly(o.flatten(1, 2).transpose(1, 2).contiguous(), c["had"])
    return _packed(s, o).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "prompt": _plain_prompt, "tree": _plain_tree, "move": _plain_move}[op](s)
    import int4_weight_kv_gb300 as ft

    c = s["case"]
    if op == "qk":
        ft.check(ft.ft_qk_norm_rope_bf16(s["cfg"], s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["total"], s["q_out"], s["k_out"]),
                 "ft_qk_norm_rope_bf16")
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        ft.check(ft.ft_kv_append_rope_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["k"], s["v"], s["gk"], s["pos"],
                                                 s["slots"], s["total"], s["q"], s["gq"], s["q_out"]), "ft_kv_append_rope_paged_int4")
        ft.check(ft.ft_kv_read_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["slots"], s["total"], s["k_out"], s["v_out"]),
                 "ft_kv_read_paged_int4")
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if op == "prompt":
        ft.check(ft.ft_attn_prompt_bf16(s["cfg"], s["q"], s["k"], s["v"], s["cu"], s["B"], s["total"], s["max"], c["d"] ** -0.5, s["o"]),
                 "ft_attn_prompt_bf16")
        return s["o"]
    if op == "tree":
        ft.check(ft.ft_attn_tree_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["q"], s["cu"], s["kv_len"], s["table"],
                                            s["mask"], s["B"], s["total"], s["max_q"], c["d"] ** -0.5, s["o"], s["ws"]),
                 "ft_attn_tree_paged_int4")
        return s["o"]
    ft.check(ft.ft_kv_move_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["src"], s["dst"]), "ft_kv_move_paged_int4")
    return s["pool"]


# ------------------------------------------------------------------ 64 bits
def _sylvester(n):
    i = torch.arange(n, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = sum(((bits >> b) & 1) for b in range(8)) % 2
    return (1.0 - 2.0 * odd.double()) / math.sqrt(n)


def _rotate64(x, block):
    x = x.double()
    return (x.reshape(-1, block) @ _sylvester(block)).reshape(x.shape)


def _turn64(x, gain, pos):
    """Norm and rotation by complex multiplication, in 64 bits."""
    x, d = x.double(), x.shape[-1]
    if gain is not None:
        x = gain.double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    freq = torch.exp(torch.arange(d // 2, device="cuda", dtype=torch.float64) * (-2 / d * math.log(BASE)))
    ang = pos.double()[:, None, None] * freq
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(ang), ang)
    return torch.cat((z.real, z.imag), -1)


def _entries64(block, page, d):
    """Values of one request's pages, uint8 [n, page (d + 4)], channel by channel from the layout's definition."""
    by = block.to(torch.int64)
    pos, ch = torch.arange(page, device="cuda")[:, None], torch.arange(d, device="cuda")[None, :]
    j, e, g = ch // 32, (ch // 8) % 4, ch % 8
    pair = pos // 2
    turn = 2 * (pair % 4) if d == 128 else 4 * ((pair // 2) % 2)
    at = {"k": pos * (d // 2) + (g // 2) * (d // 8) + 4 * j + 2 * (g % 2),
          "v": page * d // 2 + pair * d + (g ^ turn) * (d // 8) + 4 * j + 2 * (pos % 2)}
    mag, sgn = torch.tensor(MAG, device="cuda")[e], torch.tensor(SGN, device="cuda")[e]
    got = []
    for n, name in enumerate(("k", "v")):
        w = by[:, at[name]] + 256 * by[:, at[name] + 1]
        q = ((w >> mag) & 7) * (1 - 2 * ((w >> sgn) & 1))
        where = page * d + 4 * torch.arange(page, device="cuda") + 2 * n
        raw = by[:, where] + 256 * by[:, where + 1]
        scale = (raw << 16).to(torch.int32).view(torch.float32).double()
        got.append((q.double() * scale[..., None]).flatten(0, 1))
    return got


def exact(case, seed):
    op = case["op"]
    if op == "move":
        return None
    s = prepare(case, seed)
    if op == "qk":
        return {"q": _turn64(s["q"], s["gq"], s["pos"]), "k": _turn64(s["k"], s["gk"], s["pos"])}
    if op == "append":
        out = {"q": _turn64(s["q"], s["gq"], s["pos"])}
        for name, x in (("k", _turn64(s["k"], s["gk"], s["pos"])), ("v", s["v"])):
            r = _rotate64(x, case["had"])
            scale = (r.abs().amax(-1, keepdim=True).float() / 7).to(torch.bfloat16).double()
            code = torch.where(scale > 0, torch.round(r / scale.clamp(min=1e-300)), torch.zeros_like(r)).clamp(-7, 7)
            out[name] = _rotate64(code * scale, case["had"])
        return out
    d, h = case["d"], case["n_kv"]
    group = case["n_q"] // h
    new, kv = lengths(case)
    if work(case)["flops"] > 4e12:
        return None
    out = torch.empty((s["total"], case["n_q"], d), dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        rows = slice(first, first + n)
        if op == "prompt":
            hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        else:
            pages = s["table"][b, :-(-length // case["page"])].long()
            see = [[False] * n for _ in range(n)]
            for i, up in enumerate(trees(case)[b]):
                see[i] = list(see[up]) if up >= 0 else [False] * n
                see[i][i] = True
            hidden = torch.cat((torch.zeros((n, length - n), dtype=torch.bool), ~torch.tensor(see)), 1).cuda()
        for i in range(h):
            if op == "prompt":
                k, v = s["k"][rows, i].double(), s["v"][rows, i].double()
            else:
                k, v = (t[:length] for t in _entries64(s["pool"][pages, i], case["page"], d))
            for x in range(i * group, (i + 1) * group):
                q = s["q"][rows, x].double() if op == "prompt" else _rotate64(s["q"][rows, x], case["had"])
                o = torch.softmax((q @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf), -1) @ v
                out[rows, x] = o if op == "prompt" else _rotate64(o, case["had"])
        first += n
    return out
