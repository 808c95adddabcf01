"""Paged 4-bit KV cache and token log probabilities (oracle; test infrastructure only).

The cache's rotation and quantiser are those of kv.py (summary page, "무엇과
다른가"); the pages that requests share, the slot map and the log probabilities
are this library's own calls.  Everything is evaluated in FP64 with plain NumPy;
the page layout is read word by word from its definition in include/ft.h.
"""
import numpy as np

from .hadamard import blockdiag_apply
from .rope import rope_apply


def page_map(page_size, ctx, new, table, free, head=0, n_slots=None):
    """The step's map, request by request: dict of cu, kv_len, table, slots, head, capacity (a request was not served)."""
    B, out = len(ctx), np.array(table, np.int64)
    cu = np.concatenate([[0], np.cumsum([max(int(n), 0) for n in new])])
    n_slots = int(cu[-1]) if n_slots is None else n_slots
    slots = np.full(n_slots, -1, np.int64)
    kv = np.zeros(B, np.int64)
    asked, taken, short = 0, 0, False
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        if c < 0 or n < 0 or c + n > out.shape[1] * page_size:
            short = True
            continue
        old, need = -(-c // page_size), -(-(c + n) // page_size)
        if need > old:
            first, asked = asked, asked + need - old
            if asked > len(free) - head:
                short = True
                continue
            out[b, old:need] = free[head + first:head + asked]
            taken = asked
        kv[b] = c + n
        for i in range(n):
            if cu[b] + i < n_slots:
                slots[cu[b] + i] = out[b, (c + i) // page_size] * page_size + (c + i) % page_size
    return {"cu": cu, "kv_len": kv, "table": out, "slots": slots, "head": head + taken, "capacity": short}


def unpack_pages(pool, n_kv, page_size, d):
    """uint8 [n_pages, n_kv, P (d + 4)] -> codes int8 K, V [n_pages, n_kv, P, d] and FP64 scales K, V [n_pages, n_kv, P]."""
    pool = np.asarray(pool).reshape(-1, n_kv, page_size * (d + 4)).astype(np.int64)
    mag_at, neg_at = (0, 3, 8, 11), (15, 14, 7, 6)
    k = np.zeros(pool.shape[:2] + (page_size, d), np.int8)
    v = np.zeros_like(k)
    for p in range(page_size):
        pair = p // 2
        turn = 2 * (pair % 4) if d == 128 else 4 * ((pair // 2) % 2)
        for g in range(8):
            for j in range(d // 32):
                at = (p * d // 2 + (g // 2) * (d // 8) + 4 * j + 2 * (g % 2),
                      page_size * d // 2 + pair * d + (g ^ turn) * (d // 8) + 4 * j + 2 * (p % 2))
                for dst, a in zip((k, v), at):
                    w = pool[:, :, a] | (pool[:, :, a + 1] << 8)
                    for e in range(4):
                        m = (w >> mag_at[e]) & 7
                        dst[:, :, p, 32 * j + g + 8 * e] = np.where((w >> neg_at[e]) & 1, -m, m)
    sc = pool[:, :, page_size * d:].reshape(pool.shape[:2] + (page_size, 2, 2))
    bits = ((sc[..., 0] | (sc[..., 1] << 8)) << 16).astype(np.uint32)
    s = bits.view(np.float32).astype(np.float64)
    return k, v, s[..., 0], s[..., 1]


def attend_rows(q, k_hat, v_hat, had_block, scale, first_pos):
    """q [n, d] of one query head at positions first_pos, first_pos + 1, ...; k_hat, v_hat [len, d] decoded
    entries (rotated).  Returns o [n, d] in the model basis, and for each row the sum of weight |v| (2-norm)
    and the largest |q|.|k| scale of the keys that it sees (for error bounds)."""
    n, d = q.shape
    qt = blockdiag_apply(q, had_block)
    o, vn, dn = np.zeros((n, d)), np.zeros(n), np.zeros(n)
    vlen = np.linalg.norm(v_hat, axis=-1)
    for i in range(n):
        seen = min(first_pos + i + 1, len(k_hat))
        if seen <= 0:
            continue
        s = scale * (k_hat[:seen] @ qt[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        o[i] = blockdiag_apply(w @ v_hat[:seen], had_block)
        vn[i] = w @ vlen[:seen]
        dn[i] = scale * np.max(np.abs(k_hat[:seen]) @ np.abs(qt[i]))
    return o, vn, dn


def norm_rope(x, gamma, pos, base, eps):
    """Rows x [heads, d] of one token: per-head RMS norm with gains gamma (None: none), then the rotation to pos."""
    x = np.asarray(x, np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    return rope_apply(x, int(pos), base)


def attend_seen(q, k_hat, v_hat, had_block, scale, seen):
    """q [n, d] of one query head, k_hat and v_hat [len, d] (rotated entries), seen bool [n, len].  Returns what
    attend_rows does."""
    n, d = q.shape
    qt = blockdiag_apply(q, had_block)
    o, vn, dn = np.zeros((n, d)), np.zeros(n), np.zeros(n)
    vlen = np.linalg.norm(v_hat, axis=-1)
    for i in range(n):
        j = np.nonzero(seen[i])[0]
        if not len(j):
            continue
        s = scale * (k_hat[j] @ qt[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        o[i] = blockdiag_apply(w @ v_hat[j], had_block)
        vn[i] = w @ vlen[j]
        dn[i] = scale * np.max(np.abs(k_hat[j]) @ np.abs(qt[i]))
    return o, vn, dn


def tree_rows(parents):
    """Parents of one request's drafted tokens (-1: the history) -> bool [n, n]: itself and its ancestors."""
    see = np.zeros((len(parents), len(parents)), bool)
    for i, up in enumerate(parents):
        if up >= 0:
            see[i] = see[up]
        see[i, i] = True
    return see


def mask_words(see, words):
    """bool [n, m] -> int32 [n, words], bit j % 32 of word j / 32 for column j."""
    bits = np.zeros((see.shape[0], 32 * words), np.uint64)
    bits[:, :see.shape[1]] = see
    w = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def logprobs(x, targets, top):
    """FP64 logits [N, V] -> dict of logprob, entropy, rank, top_ids, top_logprobs (every row finite or -inf below)."""
    x = np.asarray(x, np.float64)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(-1, keepdims=True)
    lp = x - m - np.log(z)
    n = np.arange(len(x))
    with np.errstate(invalid="ignore"):
        ent = -np.where(e > 0, e / z * lp, 0.0).sum(-1)
    t = np.asarray(targets)
    xt = x[n, t][:, None]
    rank = ((x > xt) | ((x == xt) & (np.arange(x.shape[1])[None, :] < t[:, None]))).sum(-1)
    order = np.argsort(-x, axis=-1, kind="stable")[:, :top]
    return {"logprob": lp[n, t], "entropy": ent, "rank": rank, "top_ids": order,
            "top_logprobs": np.take_along_axis(lp, order, -1)}
