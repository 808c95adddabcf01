"""Rows of the fused projection, draft trees, moved entries and prompt attention against FP64 plain forms.

Tolerances, before any run:
* Norm and rotation.  The mean square is a sum of d positive FP32 terms, 2^-24 each and at most 20 additions deep,
  so its root and the two products are good to 2^-19 |y|.  An angle is exact to 2^-31 half turns and rounded to FP32:
  2^-25 half turns, pi 2^-25; sine and cosine add 2^-23.  |z - z64| <= 2^-18 (|y_i| + |y_(i+d/2)|) + 2^-8 |z|, the last
  the BF16 rounding.
* Codes.  With the stored scale s: a code is the nearest to z64 / s but where that is within 1e-3 of a boundary
  (2^-18 of the row's norm is under 7 sqrt(2 d) 2^-18 = 4.3e-4 of a step); a scale is amax / 7 rounded to BF16, amax
  good to 2^-17.
* Tree attention: as derived in test_paged_gpu.py.
* Prompt attention.  Products of BF16 are exact in FP32; sums of d of them, the scaling and exp2 move a score by at
  most 2^-17 max_j scale |q|.|k_j| + 2^-18 (twice, with the normaliser), each weight is rounded to BF16 (2^-8), sums
  over up to 2^13 positions lose 2^-24 each, 2^-16 in all: |o - o64| <= (2^-16 dn + 2^-8 + 2^-15) sum w |v| + 2^-8 |o|
  in the 2-norm of a row.
* Moved entries are exact.
"""
import numpy as np
import pytest
import torch

import int4_weight_kv_gb300 as ft
import oracle
from oracle import paged
from tests.test_paged_gpu import Attn, _bf16, _cfg, _gpu, _i32, _status  # noqa: F401 (_gpu: a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm and rotation
def _gain(g, d):
    x = (1 + 0.3 * g.normal(size=d)).astype(np.float32)
    return torch.from_numpy(x).cuda(), x.astype(np.float64)


def _turned(xf, gain, pos, cfg):
    """(z64, the error allowed of an FP32 z) of rows [T, heads, d]."""
    z = np.stack([paged.norm_rope(x, gain, p, cfg.rope_base, cfg.rms_eps) for x, p in zip(xf, pos)])
    y = np.abs(np.stack([paged.norm_rope(x, gain, 0, cfg.rope_base, cfg.rms_eps) for x in xf]))
    h = y.shape[-1] // 2
    both = y[..., :h] + y[..., h:]
    return z, 2.0 ** -18 * np.concatenate([both, both], -1)


def _positions(g, total, far):
    pos = g.integers(0, far, total)
    pos[0], pos[-1] = far - 1, 0
    return pos


@pytest.mark.parametrize("n_q,n_kv,d,total,pad,norm,far", [
    (32, 8, 128, 1, 0, True, 1), (32, 8, 128, 33, 16, True, 2 ** 20), (8, 2, 64, 5, 3, False, 131072), (7, 1, 128, 130, 0, True, 4096),
    (42, 6, 64, 77, 1, True, 2 ** 31), (4, 4, 128, 2, 0, False, 2 ** 31), (64, 8, 128, 1500, 16, True, 100000)])
def test_norm_rope(n_q, n_kv, d, total, pad, norm, far):
    cfg, g = _cfg(n_q, n_kv, d), np.random.default_rng(total + d)
    x, xf = _bf16(g, total, n_q + n_kv + pad, d)
    x[0, 0], xf[0, 0] = 0, 0                                                       # a row of zeros
    (gq, gqf), (gk, gkf) = (_gain(g, d), _gain(g, d)) if norm else ((None, None), (None, None))
    pos = _positions(g, total, far)
    q, k = x[:, pad:pad + n_q], x[:, pad + n_q:]
    out = torch.full((total + 1, n_q + n_kv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, q, k, gq, gk, _i32(pos), total, out[:, :n_q], out[:, n_q:]))
    got = out.float().cpu().numpy().astype(np.float64)
    assert (got[total] == 7.0).all()
    for lo, hi, gain, src in ((0, n_q, gqf, xf[:, pad:pad + n_q]), (n_q, n_q + n_kv, gkf, xf[:, pad + n_q:])):
        z, tol = _turned(src, gain, pos, cfg)
        # at 2^31 the frequencies' own 64-bit fractions are 2^-33 of a turn off, nothing beside the rest
        assert np.all(np.abs(got[:total, lo:hi] - z) <= tol + 2.0 ** -8 * np.abs(z))
    # one of the two alone, in place, in parts at another offset: the same bits
    alone = torch.empty((total, n_kv, d), dtype=torch.bfloat16, device="cuda")
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, None, k, None, gk, _i32(pos), total, None, alone))
    assert torch.equal(alone, out[:total, n_q:])
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, q, None, gq, None, _i32(pos), total, q, None))
    assert torch.equal(q, out[:total, :n_q]) and torch.equal(x[:, pad + n_q:], k)


def test_norm_rope_odd_address_and_negative_positions():
    """Rows that start between 16-byte boundaries; positions before 0 turn the other way."""
    cfg, g = _cfg(2, 1, 128), np.random.default_rng(2)
    raw = torch.from_numpy(g.normal(size=4 * 400 + 3).astype(np.float32)).to(torch.bfloat16).cuda()
    q = raw[1:1 + 4 * 400].as_strided((4, 2, 128), (401, 128, 1), 1)
    pos = np.array([-1, -70000, 5, -2 ** 31])
    o = torch.zeros(4 * 300 + 1, dtype=torch.bfloat16, device="cuda").as_strided((4, 2, 128), (257, 128, 1), 1)
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, q, None, None, None, _i32(pos), 4, o, None))
    z, tol = _turned(q.float().cpu().numpy().astype(np.float64), None, pos, cfg)
    assert np.all(np.abs(o.float().cpu().numpy() - z) <= tol + 2.0 ** -8 * np.abs(z))


@pytest.mark.parametrize("base", [0.25, 2.0 ** -7, 1.0])
def test_norm_rope_bases_below_one(base):
    """Frequencies that grow along the channels, past a turn a position."""
    cfg, g, total = _cfg(4, 2, 64), np.random.default_rng(11), 40
    cfg.rope_base = base
    x, xf = _bf16(g, total, 6, 64)
    pos = _positions(g, total, 2 ** 16)
    out = torch.empty((total, 6, 64), dtype=torch.bfloat16, device="cuda")
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, x[:, :4], x[:, 4:], None, None, _i32(pos), total, out[:, :4], out[:, 4:]))
    z, tol = _turned(xf, None, pos, cfg)
    assert np.all(np.abs(out.float().cpu().numpy() - z) <= tol + 2.0 ** -8 * np.abs(z))


# ---------------------------------------------------------------- placement on the way
def _pool(cfg, n_pages, ps, fill=0xA5):
    return torch.full((ft.ft_kv_pages_bytes(cfg, n_pages, ps),), fill, dtype=torch.uint8, device="cuda")


def _bf16_near(x):
    """Neighbours that x (1 -+ 2^-17) rounds to, as FP64."""
    return [torch.from_numpy((x * (1 + e)).astype(np.float64)).to(torch.bfloat16).double().numpy() for e in (-2.0 ** -17, 2.0 ** -17)]


@pytest.mark.parametrize("n_q,n_kv,d,had,ps,total,pad,norm", [
    (32, 8, 128, 0, 64, 70, 0, True), (8, 2, 64, 0, 16, 37, 5, False), (3, 1, 128, 32, 32, 1, 0, True), (5, 5, 128, 1, 128, 130, 2, False),
    (42, 6, 64, 16, 16, 333, 1, True), (4, 4, 64, 2, 64, 5, 0, True), (16, 2, 128, 64, 16, 2100, 0, True), (8, 8, 128, 4, 32, 9, 0, False),
    (2, 2, 64, 8, 16, 50, 0, True)])
def test_append_rope(n_q, n_kv, d, had, ps, total, pad, norm):
    cfg, g = _cfg(n_q, n_kv, d, had), np.random.default_rng(d + total)
    n_pages = -(-total // ps) + 2
    x, xf = _bf16(g, total, pad + n_q + 2 * n_kv, d)
    x[0], xf[0] = 0, 0
    x[total // 2] *= 2.0 ** 20
    xf[total // 2] *= 2.0 ** 20
    q, k, v = x[:, pad:pad + n_q], x[:, pad + n_q:pad + n_q + n_kv], x[:, pad + n_q + n_kv:]
    (gq, _), (gk, gkf) = (_gain(g, d), _gain(g, d)) if norm else ((None, None), (None, None))
    slots = g.permutation(n_pages * ps)[:total]
    if total > 40:
        slots[:32] = np.arange(32) + 2                                             # runs of neighbours, as a prompt's
    slots = np.array(list(dict.fromkeys(slots.tolist())) + [-1] * total)[:total]
    if total > 2:
        slots[total // 3] = -1
    pos = _positions(g, total, 50000)
    pool, st, qo = _pool(cfg, n_pages, ps), _status(), torch.empty((total, n_q, d), dtype=torch.bfloat16, device="cuda")
    ft.check(ft.ft_kv_append_rope_paged_int4(cfg, pool, n_pages, ps, k, v, gk, _i32(pos), _i32(slots), total, q, gq, qo, st))
    assert ft.ft_read_device_status(st) == 0
    # the queries' bits are the other call's; without queries the pool's are the same
    want = torch.empty_like(qo)
    ft.check(ft.ft_qk_norm_rope_bf16(cfg, q, None, gq, None, _i32(pos), total, want, None))
    assert torch.equal(qo, want)
    pool2 = _pool(cfg, n_pages, ps)
    ft.check(ft.ft_kv_append_rope_paged_int4(cfg, pool2, n_pages, ps, k, v, gk, _i32(pos), _i32(slots), total))
    assert torch.equal(pool, pool2)
    # V's codes and scales, and entries that no slot names, are those of the placement without rotation
    plain = _pool(cfg, n_pages, ps)
    ft.check(ft.ft_kv_append_paged_int4(cfg, plain, n_pages, ps, k, v, _i32(slots), total))
    a, b = (paged.unpack_pages(t.cpu().numpy(), n_kv, ps, d) for t in (pool, plain))
    for i in (1, 3):
        np.testing.assert_array_equal(a[i], b[i])
    on = slots >= 0
    there = np.zeros(n_pages * ps, bool)
    there[slots[on]] = True
    idle = (~there).reshape(n_pages, ps).nonzero()
    for i in (0, 2):
        np.testing.assert_array_equal(a[i][idle[0], :, idle[1]], b[i][idle[0], :, idle[1]])
    pg, of = slots[on] // ps, slots[on] % ps
    codes, s = a[0][pg, :, of], a[2][pg, :, of]
    z, _ = _turned(xf[:, pad + n_q:pad + n_q + n_kv], gkf, pos, cfg)
    r = oracle.blockdiag_apply(z[on], had or d)
    lo, hi = _bf16_near(np.abs(r).max(-1) / 7)
    assert np.all((s >= lo) & (s <= hi))
    t = r / np.where(s == 0, 1, s)[..., None]
    off = np.abs(codes - np.clip(t, -7, 7))
    assert np.all(off <= 0.5 + 1e-3) and not codes[s == 0].any()
    # positions 0 and no norm: the same pool as without rotation, bit for bit
    pool3 = _pool(cfg, n_pages, ps)
    ft.check(ft.ft_kv_append_rope_paged_int4(cfg, pool3, n_pages, ps, k, v, None, _i32(pos * 0), _i32(slots), total))
    assert torch.equal(pool3, plain)


def test_append_rope_flags():
    cfg = _cfg(2, 2, 64)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for slots, bad in (([0, 32, 1], True), ([0, -2, 1], True), ([3, 31, -1], False)):
        pool, st, ref = _pool(cfg, 2, 16), _status(), _pool(cfg, 2, 16)
        ft.check(ft.ft_kv_append_rope_paged_int4(cfg, pool, 2, 16, x, x, None, _i32([0, 0, 0]), _i32(slots), 3, dev_status=st))
        assert ft.ft_read_device_status(st) == (ft.FT_DEV_RANGE if bad else 0)
        ft.check(ft.ft_kv_append_paged_int4(cfg, ref, 2, 16, x, x, _i32(slots), 3))
        assert torch.equal(pool, ref)
    for which in (0, 1):
        y = x.clone()
        y[1, 1, 5] = float("nan")
        st = _status()
        ft.check(ft.ft_kv_append_rope_paged_int4(cfg, _pool(cfg, 2, 16), 2, 16, y if which == 0 else x, x if which == 0 else y, None,
                                                 _i32([5, 6, 7]), _i32([4, 5, 6]), 3, dev_status=st))
        assert ft.ft_read_device_status(st) == ft.FT_DEV_RANGE


# ---------------------------------------------------------------- moved entries
@pytest.mark.parametrize("n_kv,d,ps,B,n", [(8, 128, 64, 3, 5), (2, 64, 16, 1, 1), (6, 64, 32, 40, 13), (2, 128, 16, 2, 256), (3, 128, 128, 9, 64)])
def test_move(n_kv, d, ps, B, n):
    """Overlapping moves of one request happen at once; -1 on either side and equal slots change nothing."""
    cfg, g = _cfg(n_kv, n_kv, d), np.random.default_rng(n + d)
    per = -(-2 * n // ps) + 1                                                        # pages of a request
    n_pages = B * per + 1
    raw = torch.from_numpy(g.integers(0, 256, (ft.ft_kv_pages_bytes(cfg, n_pages, ps),), dtype=np.uint8)).cuda()
    ids = g.permutation(n_pages)[:B * per].reshape(B, per)
    src, dst = np.full((B, n), -1), np.full((B, n), -1)
    for b in range(B):
        at = np.array([ids[b, i // ps] * ps + i % ps for i in range(per * ps)])
        src[b] = at[np.sort(g.permutation(2 * n)[:n])] if b % 3 else at[g.permutation(n)]  # a branch; a permutation in place
        dst[b] = at[:n]
        if n > 4:
            src[b, n // 2], dst[b, n // 3] = -1, -1
    pool, st = raw.clone(), _status()
    ft.check(ft.ft_kv_move_paged_int4(cfg, pool, n_pages, ps, _i32(src), _i32(dst), st))
    assert ft.ft_read_device_status(st) == 0
    got, want = (list(paged.unpack_pages(t.cpu().numpy(), n_kv, ps, d)) for t in (pool, raw))
    raw_sc = lambda t: t.cpu().numpy().reshape(n_pages, n_kv, -1)[..., ps * d:].reshape(n_pages, n_kv, ps, 4)  # noqa: E731
    got[2:], want[2:] = [raw_sc(pool)], [raw_sc(raw)]                                   # the scales' bytes
    for a, b in zip(got, want):
        before = b.copy()
        for s, t in zip(src.ravel(), dst.ravel()):
            if s >= 0 and t >= 0:
                b[t // ps, :, t % ps] = before[s // ps, :, s % ps]
        np.testing.assert_array_equal(a, b)


def test_move_bad_slots():
    cfg = _cfg(2, 2, 64)
    raw = torch.arange(ft.ft_kv_pages_bytes(cfg, 2, 16), device="cuda").to(torch.uint8)
    for src, dst in (([0, 32], [1, 2]), ([0, 3], [1, -2]), ([0, 3], [1, 1 << 30])):
        pool, st = raw.clone(), _status()
        ft.check(ft.ft_kv_move_paged_int4(cfg, pool, 2, 16, _i32([src]), _i32([dst]), st))
        assert ft.ft_read_device_status(st) == ft.FT_DEV_RANGE
        ref = raw.clone()
        ft.check(ft.ft_kv_move_paged_int4(cfg, ref, 2, 16, _i32([[0]]), _i32([[1]])))
        assert torch.equal(pool, ref)


# ---------------------------------------------------------------- draft trees
class Tree(Attn):
    """An Attn problem whose new tokens see each other by a mask: "tree", "causal", "none", "all" or "random"."""

    def __post_init__(self):
        self.kind = self.__dict__.pop("kind", "tree")
        super().__post_init__()
        self.masks()

    def masks(self, kind=None, extra=0):
        kind, g = kind or self.kind, np.random.default_rng(self.seed + self.total)
        self.see = []
        for n in self.qlens:
            if kind == "tree":
                see = paged.tree_rows([int(g.integers(max(-1, i - 4), i)) for i in range(n)])
            elif kind == "random":
                see = g.random((n, n)) < 0.5
            else:
                see = {"causal": np.tril, "all": np.ones_like, "none": np.zeros_like}[kind](np.ones((n, n), bool))
            self.see.append(see)
        words = -(-max(max(self.qlens), 1) // 32) + extra
        rows = [paged.mask_words(s, words) for s in self.see if len(s)]
        if kind != "causal":                                                         # bits of tokens that are not there
            for r, s in zip(rows, [s for s in self.see if len(s)]):
                full = paged.mask_words(np.concatenate([np.zeros_like(s), np.ones((len(s), 32 * words - s.shape[1]), bool)], 1), words)
                r |= full
        self.mask = torch.from_numpy(np.concatenate(rows)).cuda()

    def run(self, max_q=None, ws=None, stream=None, o=None, status=None, q=None):
        o = torch.full((self.total + 2, self.n_q, self.d), 7.0, dtype=torch.bfloat16, device="cuda") if o is None else o
        max_q = max(max(self.qlens) if max_q is None else max_q, 1)
        st = _status() if status is None else status
        if ws is None:
            ws = torch.full((ft.ft_attn_tree_workspace_bytes(self.cfg, self.B, self.total, max_q),), 0xFF, dtype=torch.uint8, device="cuda")
        ft.check(ft.ft_attn_tree_paged_int4(self.cfg, self.pool, self.n_pages, self.ps, self.q if q is None else q, _i32(self.cu),
                                            _i32(self.kvlens), _i32(self.table), self.mask, self.B, self.total, max_q, self.scale, o, ws,
                                            st, stream))
        torch.cuda.synchronize()
        return o, int(st.item())

    def check(self, o, reqs=None, heads=None, floor=2.0 ** -35):
        G = self.n_q // self.n_kv
        got = o.float().cpu().numpy().astype(np.float64)
        assert (got[self.total:] == 7.0).all()
        k, v, ks, vs = paged.unpack_pages(self.pool_np, self.n_kv, self.ps, self.d)
        for b in range(self.B) if reqs is None else reqs:
            n, kv = self.qlens[b], self.kvlens[b]
            if not n:
                continue
            pages, seen = self.table[b, :-(-kv // self.ps)], np.zeros((n, kv), bool)
            seen[:, :max(kv - n, 0)] = True
            new = min(n, kv)                                                           # tokens that have an entry: the last ones
            seen[:, kv - new:] = self.see[b][:, n - new:]
            for h in range(self.n_q) if heads is None else heads:
                j = h // G
                kh, vh = (c[pages, j].reshape(-1, self.d)[:kv] * s[pages, j].reshape(-1, 1)[:kv] for c, s in ((k, ks), (v, vs)))
                rows = slice(self.cu[b], self.cu[b] + n)
                o64, vn, dn = paged.attend_seen(self.qf[rows, h], kh, vh, self.had or self.d, self.scale, seen)
                err = np.linalg.norm(got[rows, h] - o64, axis=-1)
                tol = (2.0 ** -10 * dn + 2.0 ** -11 + 2.0 ** -16) * vn + 2.0 ** -8 * np.linalg.norm(o64, axis=-1)
                tol += kv * floor * vs[pages, j].reshape(-1)[:kv].max(initial=0.0) * 7 * self.d ** 0.5
                assert not got[rows, h][vn == 0].any()
                assert (err <= tol).all(), (b, h, float(np.max(err / np.maximum(tol, 1e-300))))


TREES = [
    # single tokens and small trees of every width of the first kernel; page and tile edges
    ((8, 2, 64, 16, [1], [1]), "tree"), ((32, 8, 128, 64, [7] * 5, [7, 8, 70, 64, 400]), "tree"), ((32, 8, 128, 64, [2, 1, 2], [63, 65, 700]), "tree"),
    ((64, 8, 128, 16, [4, 0, 3], [68, 5, 1000]), "random"), ((12, 4, 128, 128, [5, 9], [127, 300]), "tree"), ((4, 4, 64, 32, [32, 17], [90, 40]), "all"),
    # trees of many rows: a word of the mask, several, ends inside a word, masks across tiles
    ((32, 8, 128, 64, [64], [1500]), "tree"), ((8, 2, 64, 16, [33, 1, 65, 130], [33, 50, 65, 1000]), "tree"), ((64, 8, 128, 64, [48, 31], [1500, 31]), "random"),
    ((42, 6, 64, 64, [90, 40], [217, 40]), "tree"), ((7, 1, 128, 16, [259], [640]), "tree"), ((16, 2, 128, 32, [129, 0, 17], [129, 10, 400]), "all"),
    ((6, 2, 128, 128, [100, 200], [357, 200]), "random"), ((8, 8, 128, 16, [96, 1, 300], [1000, 1, 333]), "tree"),
    # masks that leave rows empty, with and without a history; tokens before position 0
    ((8, 2, 64, 16, [5, 3], [5, 30]), "none"), ((32, 8, 128, 64, [70, 40], [70, 90]), "none"), ((8, 2, 64, 16, [5, 3, 1], [2, 0, 0]), "random"),
    ((8, 2, 128, 64, [150, 90], [70, 0]), "random"), ((32, 8, 128, 64, [6, 40], [6, 900]), "random"),
    # causal masks
    ((32, 8, 128, 64, [8], [300]), "causal"), ((8, 2, 64, 32, [100, 7], [250, 90]), "causal"),
]


def _tree(i, **more):
    t = Tree.__new__(Tree)
    t.kind = TREES[i][1]
    Tree.__init__(t, *TREES[i][0], **more)
    return t


@pytest.mark.parametrize("i", range(len(TREES)))
def test_tree(i):
    a = _tree(i)
    o, st = a.run()
    assert st == 0
    a.check(o)
    o2, _ = a.run()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("i", [1, 6])
def test_tree_bounds_strides_and_place(i):
    """A larger max_q (perhaps another kernel), masks with room behind them, o over q: the same rows."""
    a = _tree(i, pad=4)
    want, _ = a.run()
    a.check(want)
    a.masks(extra=3)
    o, st = a.run()
    assert st == 0 and torch.equal(o, want)
    buf = a.q.clone()
    o, _ = a.run(o=buf, q=buf)
    assert torch.equal(o[:a.total], want[:a.total])
    o, st = a.run(max_q=max(a.qlens) + 60)
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("i", [1, 6, 12])
def test_tree_workspace_at_16_bytes(i):
    """A workspace at an odd multiple of 16 bytes, of just the size asked for."""
    a = _tree(i)
    want, _ = a.run()
    size = ft.ft_attn_tree_workspace_bytes(a.cfg, a.B, a.total, max(a.qlens))
    buf = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    at = 16 + (-buf.data_ptr()) % 32
    o, st = a.run(ws=buf[at:at + size])
    assert st == 0 and torch.equal(o, want)
    assert (buf[:at] == 0xFF).all() and (buf[at + size:] == 0xFF).all()


@pytest.mark.parametrize("heads,qlens,kvlens", [(64, [64], [20000]), (32, [7] * 3, [9000, 33000, 40]), (32, [24, 24], [12000, 5000])])
def test_tree_long(heads, qlens, kvlens):
    a = Tree(heads, 8, 128, 64, qlens, kvlens)
    o, st = a.run()
    assert st == 0
    a.check(o, heads=[0, heads // 2 + 1, heads - 1])


@pytest.mark.parametrize("qlens", [[3, 2, 4], [6, 2, 7], [40, 2, 60]])
def test_tree_bad_requests(qlens):
    a = Tree(8, 2, 128, 16, qlens, [50, 70, 90])
    want, _ = a.run()
    a.table[1, 2] = a.n_pages
    o, st = a.run()
    assert st == ft.FT_DEV_RANGE
    a.check(o, reqs=[0, 2])
    a.table[1, 2] = 0
    a.kvlens[1] = -4
    o, st = a.run()
    assert st == ft.FT_DEV_CAPACITY and not o[a.cu[1]:a.cu[2]].any()
    a.check(o, reqs=[0, 2])
    a.kvlens[1] = 70
    cu = a.cu.copy()
    a.cu = np.array([0, cu[1], cu[1] - 1, cu[1] - 1])
    o, st = a.run()
    assert st == ft.FT_DEV_RANGE and torch.equal(o[:cu[1]], want[:cu[1]]) and (o[cu[1]:] == 7.0).all()
    a.cu = np.array([0, cu[1], cu[2], a.total + 1])
    o, st = a.run(max_q=max(qlens) + 1)
    assert st == ft.FT_DEV_RANGE and (o[cu[2]:] == 7.0).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 2.0 ** 13])
@pytest.mark.parametrize("n,d", [(5, 128), (5, 64), (3, 128), (100, 128), (100, 64)])
def test_tree_entries_that_a_row_does_not_see(n, d, what):
    """A new token's entry with scales that are not finite, or far above its neighbours', is not there for rows whose masks
    leave it out."""
    a = Tree(32, 8, d, 64, [n, n], [n + 60, n + 60])
    bad = n // 2
    for s in a.see:
        s[:, bad] = False
    words = a.mask.shape[1]
    a.mask = torch.from_numpy(np.concatenate([paged.mask_words(s, words) for s in a.see])).cuda()
    a.set_scales(0, [60 + bad], k=what, v=what)
    o, st = a.run()
    k = a.pool_np.copy()
    a.set_scales(0, [60 + bad], k=0.5, v=0.5)                                           # the oracle's: any finite one
    a.check(o, floor=2.0 ** -27)
    assert k is not None


@pytest.mark.parametrize("k,v", [(float("nan"), 0.5), (0.5, float("nan")), (float("inf"), 0.5), (0.5, float("inf")), (2.0 ** 111, 0.5), (0.5, 2.0 ** 111),
                                 (float("nan"), float("inf"))])
@pytest.mark.parametrize("n,d", [(3, 128), (3, 64), (5, 128), (5, 64), (100, 128), (100, 64)])
def test_tree_entries_that_some_rows_see(n, d, k, v):
    """A new token's entry with a scale that is not finite, or 2^110 and more: the rows whose masks name it are NaN, those
    beside them are as they would be with any other entry there, and the status says nothing."""
    a = Tree(32, 8, d, 64, [n, n], [n + 60, n + 60])
    bad, sees = n // 2, np.arange(n) % 2 == 1
    for s in a.see:
        s[:, bad] = sees
    words = a.mask.shape[1]
    a.mask = torch.from_numpy(np.concatenate([paged.mask_words(s, words) for s in a.see])).cuda()
    a.set_scales(0, [60 + bad], k=0.5, v=0.5)
    fine, st = a.run()
    assert st == 0
    a.set_scales(0, [60 + bad], k=k, v=v)
    o, st = a.run()
    assert st == 0
    rows = torch.from_numpy(np.nonzero(sees)[0]).cuda()
    assert torch.isnan(o[rows].float()).all()
    a.set_scales(0, [60 + bad], k=0.5, v=0.5)                                           # the oracle's
    o[rows] = fine[rows]
    a.check(o)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("n", [1, 4, 7, 40])
def test_tree_rows_of_no_request(n, what):
    """Rows before the first request's and behind the last one's (a call padded to a fixed number of rows) may hold
    anything: nothing is reported and nothing written.  The same in a request's row is reported."""
    a = Tree(8, 2, 128, 16, [n, n], [n + 150, n + 20])
    want, st = a.run()
    assert st == 0
    rows, front, end = a.total, 3, 4
    pad = lambda t, x, top, low: torch.cat([torch.full((top, *t.shape[1:]), x, dtype=t.dtype, device="cuda"), t,  # noqa: E731
                                            torch.full((low, *t.shape[1:]), x, dtype=t.dtype, device="cuda")])
    a.total, a.cu = rows + front + end, a.cu + front
    a.q, a.mask = pad(a.q[:rows], what, front, end), pad(a.mask, -1, front, end)
    o, st = a.run(max_q=n)
    assert st == 0
    assert torch.equal(o[front:front + rows], want[:rows]) and (o[:front] == 7.0).all() and (o[front + rows:] == 7.0).all()
    a.q[front + rows - 1, 3] = what
    o, st = a.run(max_q=n)
    assert st == ft.FT_DEV_RANGE and torch.equal(o[front:front + n], want[:n])


@pytest.mark.parametrize("B", [40, 300])
def test_tree_many_requests_of_many_rows(B):
    """Batches of trees of 33 rows and more with d = 128, some without tokens."""
    g = np.random.default_rng(B)
    qlens = np.where(g.random(B) < 0.2, 0, g.integers(1, 25, B))
    qlens[-1] = 24
    a = Tree(32, 8, 128, 64, qlens.tolist(), (qlens + g.integers(0, 300, B)).tolist())
    o, st = a.run()
    assert st == 0
    a.check(o, reqs=sorted({*range(0, B, max(B // 20, 1)), B - 2, B - 1}), heads=[0, 13, 31])


@pytest.mark.parametrize("n", [3, 7, 24])
@pytest.mark.parametrize("B", [31, 32, 33, 1024, 1100])
def test_tree_many_requests(B, n):
    """Trees of every size up to n, none in many: the shares find their requests however many there are."""
    g = np.random.default_rng(B + n)
    qlens = np.where(g.random(B) < 0.4, 0, g.integers(0, n + 1, B))
    qlens[-1] = n
    a = Tree(8, 2, 64, 16, qlens.tolist(), (qlens + g.integers(0, 40, B)).tolist())
    o, st = a.run()
    assert st == 0
    a.check(o, reqs=sorted({*range(0, B, max(B // 20, 1)), B - 2, B - 1}))


@pytest.mark.parametrize("n,d", [(3, 128), (7, 128), (7, 64), (40, 128), (40, 64)])
@pytest.mark.parametrize("down", [False, True])
def test_tree_scores_that_rise(n, d, down):
    """Each 64 positions' scores 1.3 times those before (behind) them: the running maximum moves at every tile, or at none."""
    a = Tree(8, 2, d, 64, [n, n], [1500, 900])
    for b, kv in enumerate(a.kvlens):
        for i in range(0, kv, 64):
            a.set_scales(b, range(i, min(i + 64, kv)), k=0.02 * 1.3 ** ((kv - i if down else i) // 64))
    o, st = a.run()
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("n", [1, 4, 7, 40])
def test_tree_rows_anywhere(n):
    """q and o at odd addresses and strides, nothing written between o's rows."""
    a = Tree(8, 2, 128, 16, [n, 2], [n + 150, 70])
    want, _ = a.run()
    a.q = a.q.contiguous()
    buf = torch.full((a.total * (8 * 128 + 5) + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    src = torch.zeros_like(buf)
    q, o = (t[3:].as_strided((a.total, 8, 128), (8 * 128 + 5, 128, 1)) for t in (src, buf))
    q.copy_(a.q[:a.total])
    _, st = a.run(q=q, o=o)
    assert st == 0 and torch.equal(o, want[:a.total])
    o.fill_(7.0)
    assert (buf == 7.0).all()


def test_pool_beyond_4_gib():
    """Rows placed, moved and attended to on pages more than 2^32 bytes into the pool: as on its first pages."""
    cfg, ps, n_pages, few = _cfg(8, 2, 128), 64, 2 ** 32 // (2 * 64 * 132) + 40, 20
    big = torch.empty(ft.ft_kv_pages_bytes(cfg, n_pages, ps), dtype=torch.uint8, device="cuda").view(n_pages, -1)
    g, base = np.random.default_rng(2), n_pages - few
    assert base * big.shape[1] > 2 ** 32
    x, _ = _bf16(g, 1000, 4, 128)
    slots = g.permutation(few * ps)[:1000]
    small = torch.zeros((few, big.shape[1]), dtype=torch.uint8, device="cuda")
    big[base:] = 0
    src, dst = slots[:100].reshape(2, 50), np.setdiff1d(np.arange(few * ps), slots)[:100].reshape(2, 50)
    for pool, pages, at in ((small, few, 0), (big, n_pages, base)):
        st = _status()
        ft.check(ft.ft_kv_append_rope_paged_int4(cfg, pool.view(-1), pages, ps, x[:, :2], x[:, 2:], None, _i32(np.arange(1000)), _i32(slots + at * ps), 1000,
                                                 dev_status=st))
        ft.check(ft.ft_kv_move_paged_int4(cfg, pool.view(-1), pages, ps, _i32(src + at * ps), _i32(dst + at * ps), st))
        assert ft.ft_read_device_status(st) == 0
    assert torch.equal(big[base:], small) and small.any()
    for n in (2, 7, 40):
        a = Tree(8, 2, 128, ps, [n, n], [600, 500])
        a.table = np.arange(20).reshape(2, 10)
        out = []
        for a.pool, a.n_pages, at in ((small.view(-1), few, 0), (big.view(-1), n_pages, base)):
            a.table = np.arange(20).reshape(2, 10) + at
            o, st = a.run()
            assert st == 0
            out.append(o)
        assert torch.equal(*out) and out[0][:a.total].any()


# ---------------------------------------------------------------- prompts
class Prompt:
    def __init__(self, n_q, n_kv, d, lens, pad=0, spread=1.0, seed=0):
        g = np.random.default_rng(seed + sum(lens) + d)
        self.cfg, self.lens, self.total, self.B = _cfg(n_q, n_kv, d), lens, sum(lens), len(lens)
        self.n_q, self.n_kv, self.d, self.scale = n_q, n_kv, d, d ** -0.5
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        x, _ = _bf16(g, self.total + 3, pad + n_q + 2 * n_kv, d)
        x[:, :pad + n_q] *= spread
        self.q, self.k, self.v = x[:, pad:pad + n_q], x[:, pad + n_q:pad + n_q + n_kv], x[:, pad + n_q + n_kv:]

    def run(self, max_len=None, o=None, q=None, status=None, stream=None):
        o = torch.full((self.total + 3, self.n_q, self.d), 7.0, dtype=torch.bfloat16, device="cuda") if o is None else o
        st = _status() if status is None else status
        ft.check(ft.ft_attn_prompt_bf16(self.cfg, self.q if q is None else q, self.k, self.v, _i32(self.cu), self.B, self.total,
                                        max(self.lens) if max_len is None else max_len, self.scale, o, st, stream))
        torch.cuda.synchronize()
        return o, int(st.item())

    def check(self, o, seqs=None, heads=None, rows=None):
        got = o.double().cpu().numpy()
        assert (got[self.total:] == 7.0).all()
        G = self.n_q // self.n_kv
        for b in range(self.B) if seqs is None else seqs:
            a, z = self.cu[b], self.cu[b + 1]
            if a == z:
                continue
            for h in range(self.n_q) if heads is None else heads:
                q, k, v = (t[a:z, i].double() for t, i in ((self.q, h), (self.k, h // G), (self.v, h // G)))
                at = torch.arange(z - a, device="cuda") if rows is None else torch.tensor([r for r in rows if r < z - a], device="cuda")
                late = torch.arange(z - a, device="cuda")[None, :] > at[:, None]
                w = torch.softmax((q[at] @ k.T * self.scale).masked_fill(late, -torch.inf), -1)
                o64, vn = (w @ v).cpu().numpy(), (w @ v.norm(dim=-1)).cpu().numpy()
                dn = (self.scale * (q[at].abs() @ k.abs().T).masked_fill(late, 0).amax(-1)).cpu().numpy()
                err = np.linalg.norm(got[a:z, h][at.cpu().numpy()] - o64, axis=-1)
                tol = (2.0 ** -16 * dn + 2.0 ** -8 + 2.0 ** -15) * vn + 2.0 ** -8 * np.linalg.norm(o64, axis=-1)
                assert (err <= tol).all(), (b, h, float(np.max(err / np.maximum(tol, 1e-300))))


PROMPTS = [
    (8, 2, 64, [1]), (32, 8, 128, [2]), (32, 8, 128, [31, 32, 33]), (4, 4, 128, [127, 128, 129, 1]), (4, 4, 64, [255, 256, 257]),
    (64, 8, 128, [1, 0, 16, 17]), (42, 6, 64, [100, 37]), (7, 1, 128, [259, 5]), (12, 4, 128, [0, 85, 86, 0]), (10, 2, 64, [1] * 70),
    (8, 2, 64, [70, 1, 300] + [9] * 29), (8, 2, 128, [70, 1, 700] + [9] * 30),
    (32, 8, 128, [300, 1, 511, 512, 513, 77]), (8, 8, 128, [700]), (6, 2, 128, [1025, 640]), (16, 2, 64, [900, 1111]),
]


@pytest.mark.parametrize("i", range(len(PROMPTS)))
@pytest.mark.parametrize("pad", [0, 3])
def test_prompt(i, pad):
    a = Prompt(*PROMPTS[i], pad=pad)
    o, st = a.run()
    assert st == 0
    a.check(o)
    o2, _ = a.run(max_len=2 * max(a.lens) + 5)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("spread", [16.0, 1e-20, 200.0])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_sharp_and_flat(d, spread):
    a = Prompt(8, 2, d, [400, 90], spread=spread)
    o, st = a.run()
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("n_q,n_kv,d,lens", [(32, 8, 128, [5000]), (8, 2, 64, [9000, 3]), (8, 1, 128, [6001, 2000])])
def test_prompt_long(n_q, n_kv, d, lens):
    a = Prompt(n_q, n_kv, d, lens)
    o, st = a.run()
    assert st == 0
    a.check(o, heads=[0, n_q - 1], rows=list(range(0, 9000, 97)) + [lens[0] - 1])


def test_prompt_many_sequences():
    g = np.random.default_rng(4)
    a = Prompt(4, 2, 64, g.integers(0, 9, 8192).tolist())
    o, st = a.run()
    assert st == 0
    a.check(o, seqs=[0, 1, 2, 4095, 8190, 8191])


def test_prompt_in_place():
    a = Prompt(32, 8, 128, [300, 40, 129], pad=2)
    want, _ = a.run()
    buf = a.q.clone()
    o, st = a.run(o=buf, q=buf)
    assert st == 0 and torch.equal(o[:a.total], want[:a.total])


@pytest.mark.parametrize("off", [1, 2, 8])
def test_prompt_rows_anywhere(off):
    """o at any address and stride, q, k and v at strides of their own; nothing written between o's rows."""
    a = Prompt(8, 2, 128, [300, 40, 129])
    want, _ = a.run()
    a.k, a.v = a.k.contiguous(), torch.nn.functional.pad(a.v, (0, 0, 0, 3))[:, :2]
    buf = torch.full((a.total * (8 * 128 + off) + 2 * off,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[off:].as_strided((a.total, 8, 128), (8 * 128 + off, 128, 1))
    _, st = a.run(o=o)
    assert st == 0 and torch.equal(o, want[:a.total])
    o.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 60, 127, 128, 299])
def test_prompt_rows_that_are_not_finite(d, at, what):
    """A k or v that is not finite spoils the rows that see it and no other row, nor a neighbouring sequence."""
    a = Prompt(8, 2, d, [50, 300, 129])
    want, _ = a.run()
    first = int(a.cu[1])
    for t in (a.k, a.v):
        keep = t.clone()
        t[first + at, 1, 5] = what
        o, _ = a.run()
        t.copy_(keep)
        same = torch.ones(a.total, 8, dtype=torch.bool, device="cuda")
        same[first + at:a.cu[2], 4:] = False
        assert torch.equal(o[:a.total][same], want[:a.total][same])
        if t is a.v:
            assert not torch.isfinite(o[first + at:a.cu[2], 4:, 5].float()).any()
        elif not np.isinf(what):
            assert not torch.isfinite(o[first + at:a.cu[2], 4:].float()).any()
    q = a.q.clone()
    q[first + at, 3] = what
    o, _ = a.run(q=q)
    same = torch.ones(a.total, 8, dtype=torch.bool, device="cuda")
    same[first + at, 3] = False
    assert torch.equal(o[:a.total][same], want[:a.total][same])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 60, 127, 128, 299])
def test_prompt_infinite_keys(d, at):
    """An infinite value of a k: rows whose q has its sign there (a score of +infinity) are NaN, those of the other sign (a
    score of -infinity) have no weight for it."""
    a = Prompt(8, 2, d, [50, 300, 129])
    first, n = int(a.cu[1]), 300
    a.k[first + at, 1, 5] = float("inf")
    a.q[:, 4:, 5] = torch.where(torch.arange(len(a.q), device="cuda") % 2 == 0, 1.0, -1.0).to(torch.bfloat16)[:, None]
    o, st = a.run()
    assert st == 0
    a.check(o, seqs=[0, 2])
    a.check(o, seqs=[1], heads=[0, 3])
    t = torch.arange(n, device="cuda")
    up = a.q[first:first + n, 4, 5] > 0
    sees = t >= at
    alone = sees & (t == 0)                                                             # a row that sees that k only: 0 / 0
    got = o[first:first + n, 4:].double()
    assert torch.isnan(got[(sees & up) | alone]).all()
    rows = ~((sees & up) | alone)
    hidden = (t[None, :] > t[:, None]) | (t == at)[None, :] & sees[:, None]
    k, v = (x[first:first + n, 1].double() for x in (a.k, a.v))
    k[at] = 0
    for h in range(4):
        q = a.q[first:first + n, 4 + h].double()
        w = torch.softmax((q @ k.T * a.scale).masked_fill(hidden, -torch.inf), -1)
        o64, vn = w @ v, w @ v.norm(dim=-1)
        dn = a.scale * (q.abs() @ k.abs().T).masked_fill(hidden, 0).amax(-1)
        tol = (2.0 ** -16 * dn + 2.0 ** -8 + 2.0 ** -15) * vn + 2.0 ** -8 * o64.norm(dim=-1)
        assert ((got[:, h] - o64).norm(dim=-1) <= tol)[rows].all()


def test_prompt_many_blocks_of_many_sequences():
    """More than 32 prompts whose blocks are several a CTA, with d = 128."""
    g = np.random.default_rng(9)
    lens = np.where(g.random(70) < 0.1, 0, g.integers(1, 500, 70))
    lens[-1] = 499
    a = Prompt(32, 8, 128, lens.tolist())
    o, st = a.run()
    assert st == 0
    a.check(o, heads=[0, 17, 31])


def test_prompt_bad_sequences():
    a = Prompt(8, 2, 128, [50, 300, 129])
    want, _ = a.run()
    cu = a.cu.copy()
    o, st = a.run(max_len=299)
    assert st == ft.FT_DEV_RANGE and (o[50:350] == 7.0).all()
    assert torch.equal(o[:50], want[:50]) and torch.equal(o[350:], want[350:])
    for bad in ([0, 50, 49, 49], [0, 50, 350, 500], [-1, 50, 350, 479]):
        a.cu = np.array(bad)
        o, st = a.run(max_len=1000)
        assert st == ft.FT_DEV_RANGE
        fine = [b for b in range(3) if (bad[b], bad[b + 1]) == (cu[b], cu[b + 1])]
        for b in range(3):
            got = o[cu[b]:cu[b + 1]]
            assert torch.equal(got, want[cu[b]:cu[b + 1]]) if b in fine else (got == 7.0).all()


# ---------------------------------------------------------------- as a program uses them
class Drafts:
    """Steps of a serving loop that drafts trees: page map, placement with rotation, attention by the tree's mask, the kept
    branch moved to consecutive positions; the prompt before them by its own rows."""

    def __init__(self, n_q=8, n_kv=2, d=64, ps=16, prompts=(37, 5, 64), seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.cfg, self.ps, self.B, self.total0 = _cfg(n_q, n_kv, d), ps, len(prompts), sum(prompts)
        self.n_q, self.n_kv, self.d, self.prompts, self.nodes = n_q, n_kv, d, list(prompts), 9
        self.n_pages = 60
        self.pool = torch.zeros(ft.ft_kv_pages_bytes(self.cfg, self.n_pages, ps), dtype=torch.uint8, device="cuda")
        self.table, self.free, self.head = _i32(np.full((self.B, 20), -1)), _i32(np.arange(60)[::-1].copy()), _i32([0])
        self.ctx, self.st = _i32([0] * self.B), _status()
        self.parents = [-1, 0, 0, 1, 2, -1, 5, 3, 4]
        self.keep = [0, 2, 4, 8]
        see = paged.tree_rows(self.parents)
        self.depth = see.sum(1) - 1
        self.mask = torch.from_numpy(np.tile(paged.mask_words(see, 1), (self.B, 1))).cuda()
        self.gq, self.gk = (1 + 0.2 * torch.randn(d, device="cuda", generator=self.g) for _ in range(2))
        T = self.B * self.nodes
        self.rows = [torch.randn((n, n_q + 2 * n_kv, d), device="cuda", generator=self.g).to(torch.bfloat16) for n in (self.total0, T, T)]
        self.ws = torch.empty(ft.ft_attn_tree_workspace_bytes(self.cfg, self.B, T, self.nodes), dtype=torch.uint8, device="cuda")
        bf = lambda n: torch.zeros((n, n_q, d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.o, self.qb = [bf(self.total0), bf(T), bf(T)], [bf(self.total0), bf(T)]
        self.kb = torch.zeros((self.total0, n_kv, d), dtype=torch.bfloat16, device="cuda")
        self.cu0, self.cu = _i32([0] * (self.B + 1)), _i32([0] * (self.B + 1))
        self.new0, self.new, self.kv = _i32(self.prompts), _i32([self.nodes] * self.B), _i32([0] * self.B)
        self.slots0, self.slots = _i32([0] * self.total0), _i32([0] * T)
        self.pos0 = _i32(np.concatenate([np.arange(n) for n in prompts]))
        self.steps_depth, self.keep_t = _i32(np.tile(self.depth, self.B)), torch.tensor(self.keep, device="cuda")

    def run(self):
        c, n, ps = self.cfg, self.nodes, self.ps
        split = lambda x: (x[:, :self.n_q], x[:, self.n_q:self.n_q + self.n_kv], x[:, self.n_q + self.n_kv:])  # noqa: E731
        self.head.zero_(), self.ctx.zero_(), self.pool.zero_(), self.table.fill_(-1)
        ok = ft.check
        ok(ft.ft_kv_page_map(ps, self.n_pages, self.ctx, self.new0, self.B, self.table, self.free, self.head, self.head, self.cu0,
                             self.ctx, self.slots0, self.st))
        q, k, v = split(self.rows[0])
        ok(ft.ft_qk_norm_rope_bf16(c, q, k, self.gq, self.gk, self.pos0, self.total0, self.qb[0], self.kb))
        ok(ft.ft_attn_prompt_bf16(c, self.qb[0], self.kb, v, self.cu0, self.B, self.total0, max(self.prompts), self.d ** -0.5, self.o[0], self.st))
        ok(ft.ft_kv_append_rope_paged_int4(c, self.pool, self.n_pages, ps, k, v, self.gk, self.pos0, self.slots0, self.total0, dev_status=self.st))
        for step in (1, 2):
            q, k, v = split(self.rows[step])
            pos = self.ctx.repeat_interleave(n, output_size=self.B * n) + self.steps_depth
            ok(ft.ft_kv_page_map(ps, self.n_pages, self.ctx, self.new, self.B, self.table, self.free, self.head, self.head, self.cu, self.kv,
                                 self.slots, self.st))
            ok(ft.ft_kv_append_rope_paged_int4(c, self.pool, self.n_pages, ps, k, v, self.gk, pos, self.slots, self.B * n, q, self.gq, self.qb[1],
                                               self.st))
            ok(ft.ft_attn_tree_paged_int4(c, self.pool, self.n_pages, ps, self.qb[1], self.cu, self.kv, self.table, self.mask, self.B, self.B * n,
                                          n, self.d ** -0.5, self.o[step], self.ws, self.st))
            at = self.slots.view(self.B, n)
            ok(ft.ft_kv_move_paged_int4(c, self.pool, self.n_pages, ps, at[:, self.keep_t].contiguous(), at[:, :len(self.keep)].contiguous(), self.st))
            self.ctx += len(self.keep)
        return [self.pool, self.table, *self.o]


def test_drafted_steps():
    """Each step's rows are attention over what the steps before left: the prompt, then the kept branch in order."""
    a = Drafts()
    out = [t.clone() for t in a.run()]
    assert ft.ft_read_device_status(a.st) == 0
    # the second step's cache from its definition: what a program without trees would have appended in order
    pool, c, n = torch.zeros_like(a.pool), a.cfg, a.nodes
    table = out[1].cpu().numpy()
    for b, length in enumerate(a.prompts):
        first = sum(a.prompts[:b])
        rows = [a.rows[0][first + i] for i in range(length)]
        rows += [a.rows[1][b * n + i] for i in a.keep] + [a.rows[2][b * n + i] for i in a.keep]
        x = torch.stack(rows)
        pos = np.arange(len(rows))
        slots = table[b, pos // a.ps] * a.ps + pos % a.ps
        ft.check(ft.ft_kv_append_rope_paged_int4(c, pool, a.n_pages, a.ps, x[:, a.n_q:a.n_q + a.n_kv], x[:, a.n_q + a.n_kv:], a.gk, _i32(pos),
                                                 _i32(slots), len(rows)))
    got, want = (paged.unpack_pages(t.cpu().numpy(), a.n_kv, a.ps, a.d) for t in (out[0], pool))
    for b, length in enumerate(a.prompts):
        pos = np.arange(length + 2 * len(a.keep))
        for x, y in zip(got, want):
            np.testing.assert_array_equal(x[table[b, pos // a.ps], :, pos % a.ps], y[table[b, pos // a.ps], :, pos % a.ps])
    # the last row of the kept branch of step 2, as a single token behind its ancestors alone
    cu, kv = _i32(np.arange(a.B + 1)), _i32([m + 2 * len(a.keep) for m in a.prompts])
    q = a.qb[1].view(a.B, n, a.n_q, a.d)[:, a.keep[-1]].contiguous()
    o = torch.empty_like(q)
    ws = torch.empty(ft.ft_attn_paged_workspace_bytes(c, a.B, a.B, 1), dtype=torch.uint8, device="cuda")
    ft.check(ft.ft_attn_paged_int4(c, pool, a.n_pages, a.ps, q, cu, kv, a.table, a.B, a.B, 1, a.d ** -0.5, o, ws))
    # two roundings of the weights and one of each result: 2 (2^-11 + 2^-10 |score|) of values under 3 in FP16, 2^-7 of the result in BF16
    d = (out[4].view(a.B, n, a.n_q, a.d)[:, a.keep[-1]].float() - o.float()).abs()
    assert (d <= 2.0 ** -6 * 3).all() and o.float().abs().max() > 0.05


def test_drafted_steps_captured_and_without_overlap():
    want = None
    for pdl in (0, 1):
        was = ft.ft_set_pdl(pdl)
        try:
            a = Drafts(n_q=32, n_kv=8, d=128, ps=64, prompts=(130, 1, 77, 300), seed=3)
            got = [t.clone() for t in a.run()]
            if want is None:
                want = got
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                a.run()
            for _ in range(3):
                for t in a.o + [a.pool]:
                    t.fill_(0x55)
                graph.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(x, y) for x, y in zip([a.pool, a.table, *a.o], want))
            assert ft.ft_read_device_status(a.st) == 0
        finally:
            ft.ft_set_pdl(was)


@pytest.mark.parametrize("n", [2, 7, 40])
def test_captured_with_other_lengths(n):
    """A captured call reads its lengths, tables and masks when it is replayed."""
    a, p = Tree(8, 2, 128, 16, [n, n], [300, 90]), Prompt(8, 2, 128, [200, 60, 40])
    cu, kv, table, pcu = _i32(a.cu), _i32(a.kvlens), _i32(a.table), _i32(p.cu)
    o, po = torch.zeros((a.total, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((p.total, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ft.ft_attn_tree_workspace_bytes(a.cfg, 2, a.total, n), dtype=torch.uint8, device="cuda")

    def call():
        ft.check(ft.ft_attn_tree_paged_int4(a.cfg, a.pool, a.n_pages, a.ps, a.q, cu, kv, table, a.mask, 2, a.total, n, a.scale, o, ws))
        ft.check(ft.ft_attn_prompt_bf16(p.cfg, p.q, p.k, p.v, pcu, 3, p.total, 300, p.scale, po))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    a.kvlens, p.lens, p.cu = [n + 1, 64], [5, 295, 0], np.array([0, 5, 300, 300])
    kv.copy_(_i32(a.kvlens))
    pcu.copy_(_i32(p.cu))
    a.table[0, :8] = a.table[0, 7::-1].copy()
    table.copy_(_i32(a.table))
    for m in (a.mask, o, po):
        m.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = o.clone()
    want, _ = a.run(max_q=n)
    assert torch.equal(got, want[:a.total])
    want, _ = p.run(max_len=300)
    assert torch.equal(po, want[:p.total])


def test_on_another_stream():
    """The calls take the stream that they are given: nothing waits for the current one."""
    a, t = Prompt(8, 2, 128, [300, 40]), Tree(8, 2, 128, 16, [9, 3], [200, 30])
    want_p, want_t = a.run()[0], t.run()[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(a.run(stream=side)[0], want_p) and torch.equal(t.run(stream=side)[0], want_t)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, leave each other's results alone."""
    trees = [Tree(8, 2, 128, 16, [9, 3], [2000, 300], seed=1), Tree(32, 8, 128, 64, [7] * 6, [900] * 6), Tree(8, 2, 64, 16, [100, 70], [3000, 500])]
    prompts = [Prompt(8, 2, 128, [900, 40]), Prompt(8, 2, 64, [33] * 20)]
    want = [a.run()[0] for a in trees + prompts]
    got = [torch.full_like(w, 7.0) for w in want]
    ws = [torch.empty(ft.ft_attn_tree_workspace_bytes(a.cfg, a.B, a.total, max(a.qlens)), dtype=torch.uint8, device="cuda") for a in trees]
    ints = [[_i32(x) for x in ((a.cu, a.kvlens, a.table) if a in trees else (a.cu,))] for a in trees + prompts]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (a, s, o, n) in enumerate(zip(trees + prompts, streams, got, ints)):
            if i < len(trees):
                ft.check(ft.ft_attn_tree_paged_int4(a.cfg, a.pool, a.n_pages, a.ps, a.q, *n, a.mask, a.B, a.total, max(a.qlens), a.scale, o, ws[i], None, s))
            else:
                ft.check(ft.ft_attn_prompt_bf16(a.cfg, a.q, a.k, a.v, n[0], a.B, a.total, max(a.lens), a.scale, o, None, s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_arguments_of_the_wrong_kind():
    a, t = Prompt(8, 2, 128, [30]), Tree(8, 2, 128, 16, [9], [200])
    for q in (a.q.float(), a.q[:, :, ::2], a.q[:5], a.q.half()):
        with pytest.raises(ValueError):
            a.run(q=q)
    t.mask = t.mask[:, :0]
    with pytest.raises(ValueError):
        t.run()
    x, i = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda"), _i32([0] * 4)
    cfg = _cfg(2, 2, 128)
    pool = _pool(cfg, 2, 16)
    for bad in (lambda: ft.ft_qk_norm_rope_bf16(cfg, x, x, None, None, i[:3], 4, x, x), lambda: ft.ft_qk_norm_rope_bf16(cfg, x, None, None, None, i, 4, x, x),
                lambda: ft.ft_qk_norm_rope_bf16(cfg, x, None, torch.zeros(64, device="cuda"), None, i, 4, x, None),
                lambda: ft.ft_qk_norm_rope_bf16(cfg, x, None, torch.zeros(128, device="cuda").half(), None, i, 4, x, None),
                lambda: ft.ft_kv_append_rope_paged_int4(cfg, pool, 3, 16, x, x, None, i, i, 4),
                lambda: ft.ft_kv_append_rope_paged_int4(cfg, pool, 2, 16, x, x, None, i.long(), i, 4),
                lambda: ft.ft_kv_append_rope_paged_int4(cfg, pool, 2, 16, x, x, None, i, i, 4, x),
                lambda: ft.ft_kv_move_paged_int4(cfg, pool, 2, 16, i.view(2, 2), i.view(1, 4)),
                lambda: ft.ft_kv_move_paged_int4(cfg, pool, 2, 16, i, i)):
        with pytest.raises(ValueError):
            bad()
