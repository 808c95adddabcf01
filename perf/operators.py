"""Measured cases of the paged 4-bit cache operators and the token log probabilities.

Four operators of a serving step, in the order a program calls them:

* page_map:  block tables, slot maps and prefix sums from request lengths
* append:    rotate, quantise and place new K/V rows in pages of the 4-bit cache
             (the rows written are read back as values, so that they can be compared)
* attention: queries of any length per request over the paged 4-bit cache
* logprobs:  log probabilities of given tokens, entropy, rank, top alternatives

Where ``own`` is false, ``run`` computes them from elementary torch operations in
32 bits; where it is true, through the library's entry points.  ``exact`` computes
what they are defined to be in 64 bits.

A page of the cache holds, for each KV head, P positions: P K entries of d/2
bytes, P/2 V entries (one for two positions) of d bytes, and P pairs of BF16
scales (K, V).  Values are sign and magnitude (0..7), four to a 16-bit word with
channels 32 j + g + {0, 8, 16, 24}: magnitudes at bits 0, 3, 8, 11 and signs at
bits 15, 14, 7, 6.
"""
import math
import random

import torch

own = False

MAG = (0, 3, 8, 11)
SGN = (15, 14, 7, 6)
PAGE = 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 requests in mid-generation: one token each (launch latency)
        {"name": "map_step_b32", "op": "page_map", "batch": 32, "ctx": 4096, "new": 1, "page": 64, "seed": 1},
        # a batch of prompts of mixed lengths admitted at once, most of them with no history
        {"name": "map_prompts_b256", "op": "page_map", "batch": 256, "ctx": 300, "new": 2048, "page": 16, "seed": 2},
        # the new token of 32 requests of an 8B-shaped layer, K and V strided views of the fused projection
        {"name": "append_step_b32", "op": "append", "n_kv": 8, "d": 128, "had": 128, "batch": 32, "new": 1, "ctx": 4096,
         "page": 64, "fused": 32, "seed": 3},
        # prompts placed after their projection: 16 requests, 32k rows in all at most
        {"name": "append_prompts_32k", "op": "append", "n_kv": 8, "d": 128, "had": 128, "batch": 16, "new": 2048,
         "ctx": 500, "page": 32, "fused": 0, "seed": 4},
        # one request of an 8B-shaped layer, context 1024: the latency case of generation
        {"name": "attn_step_8b_b1", "op": "attention", "n_q": 32, "n_kv": 8, "d": 128, "had": 128, "batch": 1, "q": 1,
         "kv": 1025, "ragged": False, "page": 64, "fused": False, "seed": 5},
        # a serving batch of an 8B-shaped layer, requests of every length up to 4096
        {"name": "attn_step_8b_b32", "op": "attention", "n_q": 32, "n_kv": 8, "d": 128, "had": 128, "batch": 32, "q": 1,
         "kv": 4097, "ragged": True, "page": 64, "fused": True, "seed": 6},
        # long contexts of a 70B-shaped layer: eight requests of up to 32768
        {"name": "attn_step_70b_32k", "op": "attention", "n_q": 64, "n_kv": 8, "d": 128, "had": 128, "batch": 8, "q": 1,
         "kv": 32769, "ragged": True, "page": 64, "fused": False, "seed": 7},
        # prompts of a small model (head_dim 64) of odd, unequal lengths, no history
        {"name": "attn_prompts_d64", "op": "attention", "n_q": 8, "n_kv": 2, "d": 64, "had": 64, "batch": 5, "q": 777,
         "kv": 777, "ragged": True, "page": 16, "fused": False, "seed": 8},
        # a chunk of 2048 prompt tokens for each of two requests over a history of 2048
        {"name": "attn_chunk_8b_2x2048", "op": "attention", "n_q": 32, "n_kv": 8, "d": 128, "had": 128, "batch": 2,
         "q": 2048, "kv": 4096, "ragged": False, "page": 64, "fused": True, "seed": 9},
        # the next token of one request and its five best alternatives, full vocabulary
        {"name": "logprobs_b1", "op": "logprobs", "rows": 1, "vocab": 128256, "top": 5, "dtype": "f32", "pad": 0, "seed": 10},
        # a serving batch, twenty alternatives, BF16 logits with an odd vocabulary in padded rows
        {"name": "logprobs_b32_bf16", "op": "logprobs", "rows": 32, "vocab": 50257, "top": 20, "dtype": "bf16", "pad": 47,
         "seed": 11},
        # every token of a 2048-token prompt scored
        {"name": "logprobs_score_2048", "op": "logprobs", "rows": 2048, "vocab": 128256, "top": 1, "dtype": "f32", "pad": 0,
         "seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("page_map", "append", "attention", "attention", "logprobs"))
    seed, page = rng.randrange(1 << 20), rng.choice((16, 32, 64, 128))
    n_kv, g, d = rng.choice(((8, 4, 128), (8, 8, 128), (2, 4, 64), (4, 1, 128), (6, 7, 64), (4, 3, 128)))
    had = rng.choice((d, d, d, 32, 1))
    if op == "page_map":
        batch = _log(rng, 1, 512)
        new = rng.choice((1, _log(rng, 1, max(2, 262144 // batch))))
        return {"op": op, "batch": batch, "ctx": _log(rng, 1, 32768), "new": new, "page": page, "seed": seed}
    if op == "append":
        batch = _log(rng, 1, 64)
        return {"op": op, "n_kv": n_kv, "d": d, "had": had, "batch": batch, "new": rng.choice((1, _log(rng, 1, 32768 // batch))),
                "ctx": _log(rng, 1, 4096), "page": page, "fused": rng.choice((0, g * n_kv)), "seed": seed}
    if op == "attention":
        if rng.random() < 0.5:  # single tokens, or a few of them
            batch = _log(rng, 1, 64)
            q, kv = rng.choice((1, 1, 2, 5)), _log(rng, 1, min(32768, 131072 // batch))
        else:
            batch = _log(rng, 1, 8)
            q = _log(rng, 3, 2048 // batch)
            kv = q + rng.choice((0, _log(rng, 1, max(2, 4096 // batch))))
        return {"op": op, "n_q": n_kv * g, "n_kv": n_kv, "d": d, "had": had, "batch": batch, "q": q, "kv": max(kv, q),
                "ragged": rng.random() < 0.7, "page": page, "fused": rng.random() < 0.5, "seed": seed}
    rows = _log(rng, 1, 512)
    return {"op": op, "rows": rows, "vocab": _log(rng, 100, 200000), "top": rng.choice((0, 1, 5, 20, 32)),
            "dtype": rng.choice(("f32", "bf16")), "pad": rng.choice((0, 0, 5, 64)), "seed": seed}


def lengths(case):
    """(tokens to add, tokens afterwards) of each request: the longest first, then any shorter ones."""
    r, b = random.Random(case["seed"]), case["batch"]
    if case["op"] == "attention":
        new = [case["q"]] + [r.randint(1, case["q"]) if case["ragged"] else case["q"] for _ in range(b - 1)]
        kv = [case["kv"]] + [r.randint(1, case["kv"]) if case["ragged"] else case["kv"] for _ in range(b - 1)]
        return new, [max(n, k) for n, k in zip(new, kv)]
    new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(b - 1)]
    return new, [n + r.randint(0, case["ctx"]) for n in new]


def work(case):
    op = case["op"]
    if op == "logprobs":
        n, v, k = case["rows"], case["vocab"], case["top"]
        # logits read; targets, log probabilities, entropies, ranks and alternatives written
        return {"bytes": n * v * (4 if case["dtype"] == "f32" else 2) + n * (16 + 8 * k), "flops": 6.0 * n * v}
    new, kv = lengths(case)
    total, b, p = sum(new), case["batch"], case["page"]
    pages = sum(-(-k // p) for k in kv)
    if op == "page_map":
        fresh = pages - sum(-(-(k - n) // p) for n, k in zip(new, kv))
        # lengths read; prefix sums, cache lengths and slots written; new pages read and written
        return {"bytes": 4 * (2 * b + 2 * b + 1 + total + 2 * fresh), "flops": float(total)}
    d, h = case["d"], case["n_kv"]
    if op == "append":
        # BF16 rows read, entries and scales written, read again, BF16 values written
        return {"bytes": total * (4 + h * (4 * d + 2 * (d + 4) + 4 * d)), "flops": float(total * h * 2 * d * (2 * math.log2(d) + 4))}
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, kv))
    return {"bytes": sum(kv) * h * (d + 4) + 4 * total * case["n_q"] * d + 4 * pages, "flops": 4.0 * d * case["n_q"] * pairs}


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


def prepare(case, seed):
    gen, op = _gen(case, seed), case["op"]
    s = {"case": case}
    if op == "logprobs":
        n, v = case["rows"], case["vocab"]
        # logits as an LM head leaves them: a normal bulk and, row by row, more or less of a head above it
        buf = torch.randn((n, v + case["pad"]), device="cuda", generator=gen) * 2.5
        tops = torch.randint(0, v, (n, 8), device="cuda", generator=gen)
        buf.scatter_(1, tops, 8 + 8 * torch.rand((n, 8), device="cuda", generator=gen))
        buf = buf.to(torch.bfloat16) if case["dtype"] == "bf16" else buf
        pick = torch.randint(0, v, (n,), device="cuda", generator=gen)
        s["logits"] = buf[:, :v]
        s["targets"] = torch.where(torch.rand(n, device="cuda", generator=gen) < 0.7, tops[:, 0], pick).to(torch.int32)
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device="cuda")  # noqa: E731
        i = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out"] = {"logprob": f(n), "entropy": f(n), "rank": i(n)}
        if case["top"]:
            s["out"] |= {"top_ids": i(n, case["top"]), "top_logprobs": f(n, case["top"])}
        return s
    new, kv = lengths(case)
    # the largest size differs from seed to seed where only lengths are inputs
    if op == "page_map":
        drop = torch.randint(0, 2, (len(new),), generator=torch.Generator().manual_seed(seed)).tolist()
        kv = [k + x for k, x in zip(kv, drop)]
    s["total"], s["B"] = sum(new), len(new)
    s["n_pages"], table = _tables(case, kv, gen)
    s["kv_len"], s["cu"] = _ints(kv), _prefix(new)
    if op == "page_map":
        p, ctx = case["page"], [k - n for n, k in zip(new, kv)]
        old = _ints([-(-c // p) for c in ctx])
        col = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)[None, :]
        fresh = (col >= old[:, None]) & (table >= 0)
        s["free"] = torch.cat((table[fresh], torch.full((2,), s["n_pages"] - 1, dtype=torch.int32, device="cuda")))
        s["table"] = torch.where(fresh, -1, table)
        s["ctx"], s["new"], s["head"] = _ints(ctx), _ints(new), _ints([0])
        s["out"] = {"cu": torch.empty_like(s["cu"]), "kv_len": torch.empty_like(s["kv_len"]), "head": torch.empty_like(s["head"]),
                    "slots": torch.empty(s["total"], dtype=torch.int32, device="cuda"), "table": s["table"]}
        return s
    h, d = case["n_kv"], case["d"]
    s["pool"] = _pool(s["n_pages"], h, case["page"], d, gen)
    s["table"] = table
    if op == "append":
        hq = case["fused"]
        buf = torch.randn((s["total"], hq + 2 * h, d), device="cuda", generator=gen)
        hot = torch.randint(0, d, (1, hq + 2 * h, 4), device="cuda", generator=gen).expand(s["total"], -1, -1)
        buf = buf.scatter(2, hot, buf.gather(2, hot) * 20).to(torch.bfloat16)  # the outlier channels of real keys
        s["k"], s["v"] = buf[:, hq:hq + h], buf[:, hq + h:]
        req = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
        pos = torch.arange(s["total"]) - s["cu"].cpu()[req] + torch.tensor([k - n for n, k in zip(new, kv)])[req]
        req, pos, p = req.cuda(), pos.cuda(), case["page"]
        s["slots"] = (table[req, pos // p] * p + (pos % p).to(torch.int32)).contiguous()
        s["k_out"], s["v_out"] = (torch.empty((s["total"], h, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        hq = case["n_q"]
        wide = hq + 2 * h if case["fused"] else hq
        s["q"] = torch.randn((s["total"], wide, d), device="cuda", generator=gen).to(torch.bfloat16)[:, :hq]
        s["max_q"], s["max_kv"] = max(new), max(kv)
        s["o"] = torch.empty((s["total"], hq, d), dtype=torch.bfloat16, device="cuda")
    if own:
        import int4_weight_kv_gb300 as ft

        n_q = case.get("n_q") or case["n_kv"]
        s["cfg"] = ft.make_cfg(128 * n_q, n_q, case["n_kv"], d, 128, had_block=case["had"])
        if op == "attention":
            size = ft.ft_attn_paged_workspace_bytes(s["cfg"], s["B"], s["total"], s["max_q"])
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
    """BF16 rows -> int16 words [..., j, g] and BF16 scales of the rotated rows."""
    r = _butterfly(x.float(), had)
    amax = r.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).to(torch.bfloat16)
    f = s.float()[..., None]
    c = torch.where(f == 0, torch.zeros_like(r), r / torch.where(f == 0, torch.ones_like(f), f))
    c = c.round().clamp(-7, 7).to(torch.int32)
    return _halfwords(c.abs(), (c < 0).to(torch.int32)), s


def _plain_append(s):
    c, pool = s["case"], s["pool"]
    p, d, h = c["page"], c["d"], c["n_kv"]
    flat = pool.view(torch.int16).view(-1)
    slot = s["slots"].long()
    inside = slot % p
    block = ((slot // p)[:, None] * h + torch.arange(h, device="cuda")) * (p * (d + 4) // 2)  # [T, h]
    j, g = torch.arange(d // 32, device="cuda")[:, None], torch.arange(8, device="cuda")[None, :]
    k_in = (inside * (d // 4))[:, None, None] + (g >> 1) * (d // 16) + 2 * j + (g & 1)
    chunk = _chunk_of(inside >> 1, d)
    v_in = p * d // 4 + ((inside >> 1) * (d // 2))[:, None, None] + chunk[:, None, :] * (d // 16) + 2 * j + (inside & 1)[:, None, None]
    s_in = p * d // 2 + 2 * inside
    kw, ks = _quantise(s["k"], c["had"])
    vw, vs = _quantise(s["v"], c["had"])
    k_at, v_at, s_at = block[:, :, None, None] + k_in[:, None], block[:, :, None, None] + v_in[:, None], block + s_in[:, None]
    flat[k_at], flat[v_at] = kw, vw
    flat[s_at], flat[s_at + 1] = ks.view(torch.int16), vs.view(torch.int16)
    back = lambda at, e: _butterfly(_values(flat[at], flat[s_at + e].view(torch.bfloat16).float()), c["had"]).to(torch.bfloat16)  # noqa: E731
    return {"k": back(k_at, 0), "v": back(v_at, 1)}


def _plain_map(s):
    p, ctx, new, total = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["total"]
    kv = ctx + new
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    old, need = (ctx + p - 1) // p, (kv + p - 1) // p
    first = (need - old).cumsum(0) - (need - old)
    free = s["free"][s["head"].long() + torch.arange(s["free"].numel(), device="cuda")]
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    pick = free[(first[:, None] + col - old[:, None]).clamp(0, free.numel() - 1)]
    table = torch.where((col >= old[:, None]) & (col < need[:, None]), pick, s["table"])
    req = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), new, output_size=total)
    pos = torch.arange(total, device="cuda") - cu[req] + ctx[req]
    slots = table[req, pos // p] * p + pos % p
    return {"cu": cu.to(torch.int32), "kv_len": kv.to(torch.int32), "head": s["head"] + (need - old).sum().to(torch.int32),
            "slots": slots.to(torch.int32), "table": table}


def _plain_attention(s):
    c = s["case"]
    d, h, p, b, nq = c["d"], c["n_kv"], c["page"], s["B"], s["max_q"]
    g, pages = c["n_q"] // h, -(-s["max_kv"] // p)
    k, v = _decode(s["pool"][s["table"][:, :pages].clamp(min=0).long()], p, d)  # [B, pages, h, P, d]
    k, v = (t.transpose(1, 2).flatten(2, 3) for t in (k, v))  # [B, h, L, d]
    cu = s["cu"].long()
    rows = (cu[:-1, None] + torch.arange(nq, device="cuda")).clamp(max=s["total"] - 1)
    q = _butterfly(s["q"].float(), c["had"])[rows]  # [B, nq, n_q, d]
    q = q.unflatten(2, (h, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, h, g nq, d]
    sc = (q @ k.transpose(-1, -2)).unflatten(2, (g, nq)) * d ** -0.5
    n_new = cu[1:] - cu[:-1]
    pos = (s["kv_len"] - n_new)[:, None] + torch.arange(nq, device="cuda")
    seen = torch.arange(pages * p, device="cuda") <= pos[:, :, None]  # [B, nq, L]
    seen = seen & (torch.arange(pages * p, device="cuda") < s["kv_len"][:, None, None])
    sc = sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - m)
    o = (e.flatten(2, 3) @ v).unflatten(2, (g, nq)) / e.sum(-1, keepdim=True)  # [B, h, g, nq, d]
    o = _butterfly(o.permute(0, 3, 1, 2, 4).flatten(2, 3).contiguous(), c["had"])  # [B, nq, n_q, d]
    req = torch.repeat_interleave(torch.arange(b, device="cuda"), n_new, output_size=s["total"])
    return o[req, torch.arange(s["total"], device="cuda") - cu[req]].to(torch.bfloat16)


def _plain_logprobs(s):
    x, t, k = s["logits"].float(), s["targets"].long()[:, None], s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    ent = z.log() - (e * (x - m)).sum(-1, keepdim=True) / z
    lse = m + z.log()
    xt = x.gather(1, t)
    col = torch.arange(x.shape[1], device="cuda")
    out = {"logprob": (xt - lse)[:, 0], "entropy": ent[:, 0],
           "rank": ((x > xt) | ((x == xt) & (col < t))).sum(-1).to(torch.int32)}
    if k:
        val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
        out |= {"top_ids": idx[:, :k].to(torch.int32), "top_logprobs": val[:, :k] - lse}
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"page_map": _plain_map, "append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs}[op](s)
    import int4_weight_kv_gb300 as ft

    c = s["case"]
    if op == "page_map":
        o = s["out"]
        ft.check(ft.ft_kv_page_map(c["page"], s["n_pages"], s["ctx"], s["new"], s["B"], s["table"], s["free"], s["head"], o["head"],
                                   o["cu"], o["kv_len"], o["slots"]), "ft_kv_page_map")
        return o
    if op == "append":
        ft.check(ft.ft_kv_append_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["k"], s["v"], s["slots"], s["total"]),
                 "ft_kv_append_paged_int4")
        ft.check(ft.ft_kv_read_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["slots"], s["total"], s["k_out"], s["v_out"]),
                 "ft_kv_read_paged_int4")
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attention":
        ft.check(ft.ft_attn_paged_int4(s["cfg"], s["pool"], s["n_pages"], c["page"], s["q"], s["cu"], s["kv_len"], s["table"], s["B"],
                                       s["total"], s["max_q"], c["d"] ** -0.5, s["o"], s["ws"]), "ft_attn_paged_int4")
        return s["o"]
    o = s["out"]
    ft.check(ft.ft_logprobs(s["logits"], s["targets"], o["logprob"], o["entropy"], o["rank"], o.get("top_ids"), o.get("top_logprobs"),
                            c["top"]), "ft_logprobs")
    return o


# ------------------------------------------------------------------ 64 bits
def _sylvester(n):
    i = torch.arange(n, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = sum(((bits >> b) & 1) for b in range(8)) % 2
    return (1.0 - 2.0 * odd.double()) / math.sqrt(n)


def _rotate64(x, block):
    x = x.double()
    return (x.reshape(-1, block) @ _sylvester(block)).reshape(x.shape)


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
    if op == "page_map":
        return None
    s = prepare(case, seed)
    if op == "logprobs":
        parts = []
        for a in range(0, case["rows"], 64):
            x = s["logits"][a:a + 64].double()
            lp = x - torch.logsumexp(x, -1, keepdim=True)
            got = {"logprob": lp.gather(1, s["targets"][a:a + 64, None].long())[:, 0], "entropy": -(lp.exp() * lp).sum(-1)}
            if case["top"]:
                got["top_logprobs"] = lp.topk(case["top"], -1).values
            parts.append(got)
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]} | {"rank": None} | ({"top_ids": None} if case["top"] else {})
    if op == "append":
        out = {}
        for name in ("k", "v"):
            r = _rotate64(s[name], case["had"])
            scale = (r.abs().amax(-1, keepdim=True).float() / 7).to(torch.bfloat16).double()
            code = torch.where(scale > 0, torch.round(r / scale.clamp(min=1e-300)), torch.zeros_like(r)).clamp(-7, 7)
            out[name] = _rotate64(code * scale, case["had"])
        return out
    d, h, p = case["d"], case["n_kv"], case["page"]
    group = case["n_q"] // h
    new, kv = lengths(case)
    if work(case)["flops"] > 4e12:
        return None
    out = torch.empty((s["total"], case["n_q"], d), dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        pages = s["table"][b, :-(-length // p)].long()
        far = torch.arange(length, device="cuda")[None, :] > (length - n + torch.arange(n, device="cuda"))[:, None]
        for i in range(h):
            k, v = (t[:length] for t in _entries64(s["pool"][pages, i], p, d))
            for x in range(i * group, (i + 1) * group):
                sc = _rotate64(s["q"][first:first + n, x], case["had"]) @ k.T / math.sqrt(d)
                out[first:first + n, x] = _rotate64(torch.softmax(sc.masked_fill(far, -math.inf), -1) @ v, case["had"])
        first += n
    return out
