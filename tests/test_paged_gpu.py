"""The paged 4-bit cache (maps, placement, attention) and the token log
probabilities against FP64 plain forms of the same operations.

Tolerances, before any run:
* Codes follow the rule of gpu_harness.compare_codes; maps are exact.
* Attention.  Rounding q to FP16 moves a score by at most 2^-11 scale |q|.|K^|
  (half a step of each q, plus as much again for FP32 accumulation), a weight by the
  same relative amount (twice, with the normaliser); the weight itself is rounded once
  (2^-11) and taken through exp2 and log2 approximations of under 2^-18 relative.  So
  |o - o_exact| <= (2 * 2^-11 max_j scale |q|.|K^_j| + 2^-11 + 2^-16) sum_j w_j |V^_j|
  + 2^-8 |o| in the 2-norm of a row (the rotation keeps it; the last term is the BF16
  rounding).  Where the heaviest entries' values are zero the sum w |V^| says nothing of
  the weights' own floor: P = 2^10 w_j vs_j / max(w vs) has FP16's smallest step 2^-24,
  so each weight is off by up to 2^-35 max(w vs) / vs_j, and n of them move o by at most
  n 2^-35 max_j vs_j |codes| <= n 2^-35 max_j vs_j 7 sqrt(d).
* Log probabilities: a sum of V positive FP32 terms, at most V / 512 + 64 additions
  deep, each 2^-24, terms good to 2^-21, then one rounding each of x_t - lse.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from oracle import paged
import synth
import int4_weight_kv_gb300 as ft
from int4_weight_kv_gb300 import runtime as rt
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_weight_kv_gb300 import build
    build.build()


def _cfg(n_q, n_kv, d, had=0):
    return ft.make_cfg(512, n_q, n_kv, d, 512, had_block=had)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _bf16(gen, *shape):
    x = torch.from_numpy(gen.normal(0, 1, shape).astype(np.float32)).to(torch.bfloat16)
    return x.cuda(), x.float().numpy()


# ---------------------------------------------------------------- page map
def _map(ps, n_pages, ctx, new, table, free, head=0, n_slots=None, alias=False):
    B, total = len(ctx), int(np.maximum(new, 0).sum())
    n_slots = total if n_slots is None else n_slots
    c, t, h, st = _i32(ctx), _i32(table), _i32([head]), _status()
    kv = c if alias else torch.full((B,), 77, dtype=torch.int32, device="cuda")
    ho = h if alias else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    cu, slots = _i32([0] * (B + 1)), torch.full((max(n_slots, 1),), 77, dtype=torch.int32, device="cuda")[:n_slots]
    ft.check(ft.ft_kv_page_map(ps, n_pages, c, _i32(new), B, t, _i32(free), h, ho, cu, kv, slots, st))
    torch.cuda.synchronize()
    got = {"cu": cu, "kv_len": kv, "table": t, "slots": slots, "head": ho}
    return {k: v.cpu().numpy() for k, v in got.items()}, int(st.item())


@pytest.mark.parametrize("B,ps,ctx,new,alias", [(1, 16, 0, 1, False), (1, 64, 63, 1, True), (32, 64, 4000, 1, True),
                                                (7, 32, 100, 500, False), (256, 16, 300, 400, True), (1025, 128, 600, 3, False),
                                                (2, 64, 0, 9001, True), (8192, 16, 40, 2, False)])
def test_page_map(B, ps, ctx, new, alias):
    g = np.random.default_rng(B + ps)
    c, n = g.integers(0, ctx + 1, B), g.integers(0, new + 1, B)
    n[0], n[B // 2] = new, min(new, 1)
    width = int(-(-(c + n).max() // ps)) + 1
    old = -(-c // ps)
    pages = int((-(-(c + n) // ps)).sum()) + 5
    ids = g.permutation(pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :old[b]] = ids[at:at + old[b]]
        at += old[b]
    free = np.concatenate([[3, 4], ids[at:]])
    want = paged.page_map(ps, c, n, table, free, head=2, n_slots=int(n.sum()) + 9)
    got, st = _map(ps, pages, c, n, table, free, 2, int(n.sum()) + 9, alias)
    assert st == 0 and not want["capacity"]
    for k in ("cu", "kv_len", "table", "slots"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert got["head"][0] == want["head"]


@pytest.mark.parametrize("case", ["short_list", "long_row", "negative", "few_slots", "bad_page", "bad_head"])
def test_page_map_conditions(case):
    ctx, new, table, free, head, n_slots = [16, 0, 5, 3], [40, 2, 20, 0], np.full((4, 4), -1), [5, 6, 7, 8, 9], 0, None
    table[0, 0], table[2, 0], table[3, 0] = 1, 2, 3
    bit = ft.FT_DEV_CAPACITY
    if case == "short_list":
        free = free[:4]      # request 2's page is the fifth
    elif case == "long_row":
        ctx[1], new[1] = 30, 40
    elif case == "negative":
        new[0], ctx[2] = -3, -1
    elif case == "few_slots":
        n_slots, bit = 50, ft.FT_DEV_RANGE
    elif case == "bad_page":
        free[3], bit = 99, ft.FT_DEV_RANGE
    else:
        head, bit = 6, ft.FT_DEV_RANGE | ft.FT_DEV_CAPACITY
    got, st = _map(16, 10, ctx, new, table, free, head, n_slots)
    assert st == bit
    want = paged.page_map(16, ctx, new, table, free, head, n_slots)
    if case == "bad_head":
        want["head"] = 6
        assert got["kv_len"].tolist() == [0, 0, 0, 3]
    if case == "bad_page":   # request 1 asked for entry 3: its rows are dropped
        want["slots"][40:42] = -1
        want["table"][1, 0] = -1
    for k in ("cu", "kv_len", "table", "slots"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert got["head"][0] == want["head"]


# ---------------------------------------------------------------- placement
@pytest.mark.parametrize("n_kv,d,had,ps,total,fused", [(8, 128, 0, 64, 70, 32), (2, 64, 0, 16, 37, 0), (1, 128, 32, 32, 1, 3),
                                                       (5, 128, 1, 128, 130, 0), (6, 64, 16, 16, 333, 2), (4, 64, 2, 64, 5, 0)])
def test_append_codes_and_read(n_kv, d, had, ps, total, fused):
    """Same codes and scales as the dense cache's append and the oracle's quantiser; other entries untouched; the
    rows read back are the decoded entries, rotated back and rounded once."""
    cfg, g = _cfg(n_kv * 2, n_kv, d, had), np.random.default_rng(d + total)
    n_pages = -(-total // ps) + 2
    x, xf = _bf16(g, total, fused + 2 * n_kv, d)
    x[0, fused] = 0                                # an all-zero row
    xf[0, fused] = 0
    x[total // 2] *= 2.0 ** 100
    xf[total // 2] *= 2.0 ** 100
    k, v = x[:, fused:fused + n_kv], x[:, fused + n_kv:]
    slots = g.permutation(n_pages * ps)[:total]
    skip = total // 3 if total > 2 else -1
    if skip >= 0:
        slots[skip] = -1
    pool = torch.full((ft.ft_kv_pages_bytes(cfg, n_pages, ps),), 0xA5, dtype=torch.uint8, device="cuda")
    st, sl = _status(), _i32(slots)
    ft.check(ft.ft_kv_append_paged_int4(cfg, pool, n_pages, ps, k, v, sl, total, st))
    ko, vo = (torch.full((total, n_kv, d), 9, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ft.check(ft.ft_kv_read_paged_int4(cfg, pool, n_pages, ps, sl, total, ko, vo, st))
    torch.cuda.synchronize()
    assert st.item() == 0
    got = paged.unpack_pages(pool.cpu().numpy(), n_kv, ps, d)
    before = paged.unpack_pages(np.full(pool.numel(), 0xA5, np.uint8), n_kv, ps, d)
    keep = np.ones(n_pages * ps, bool)
    keep[slots[slots >= 0]] = False
    keep = keep.reshape(n_pages, ps).nonzero()
    for a, b in zip(got, before):
        np.testing.assert_array_equal(a[keep[0], :, keep[1]], b[keep[0], :, keep[1]])
    dense = rt.alloc_cache(cfg, 1, total)
    ft.check(ft.ft_kv_append_int4(cfg, dense, 1, total, k.contiguous(), v.contiguous(), _i32([0]), 1, total))
    lay = H.Layer(dataclasses.replace(synth.TINY, n_kv=n_kv, head_dim=d), cfg, {}, {})
    dk, dv, dks, dvs = H.unpack_cache(lay, dense, 1, total, 1, total)
    on = slots >= 0
    pg, of = slots[on] // ps, slots[on] % ps
    for codes, scales, dc, ds, lo, out in ((got[0], got[2], dk, dks, fused, ko), (got[1], got[3], dv, dvs, fused + n_kv, vo)):
        c, s = codes[pg, :, of], scales[pg, :, of]                      # [rows, h, d]
        np.testing.assert_array_equal(c, dc[0].transpose(1, 0, 2)[on].astype(np.int8) - 8)
        np.testing.assert_array_equal(s, ds[0, :, :, 0].T[on])
        rot = oracle.blockdiag_apply(xf[on][:, lo:lo + n_kv].astype(np.float64), had or d).astype(np.float32)
        H.compare_codes(c + 8, s.astype(np.float32)[..., None], rot, d)
        back = oracle.blockdiag_apply(c * s[..., None], had or d)
        r = out.float().cpu().numpy().astype(np.float64)
        # 7 FP32 additions and a scaling (under 2^-20 of the row's norm), then half a BF16 step
        tol = 2.0 ** -8 * np.abs(back) + 2.0 ** -20 * np.linalg.norm(back, axis=-1, keepdims=True)
        assert np.all(np.abs(r[on] - back) <= tol)
        assert skip < 0 or not r[skip].any()


def test_append_read_flags():
    cfg = _cfg(2, 2, 64)
    pool = torch.zeros(ft.ft_kv_pages_bytes(cfg, 2, 16), dtype=torch.uint8, device="cuda")
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for slots, none, bad in (([0, 32, 1], 1, True), ([0, -2, 1], 1, True), ([3, 31, -1], 2, False)):
        st = _status()
        ft.check(ft.ft_kv_append_paged_int4(cfg, pool, 2, 16, x, x, _i32(slots), 3, st))
        assert ft.ft_read_device_status(st) == (ft.FT_DEV_RANGE if bad else 0)
        ko, vo = torch.ones_like(x), torch.ones_like(x)
        st = _status()
        ft.check(ft.ft_kv_read_paged_int4(cfg, pool, 2, 16, _i32(slots), 3, ko, vo, st))
        assert ft.ft_read_device_status(st) == (ft.FT_DEV_RANGE if bad else 0)
        assert not ko[none].any() and not vo[none].any() and ko[0].any()
    y = x.clone()
    y[1, 1, 5] = float("nan")
    st = _status()
    ft.check(ft.ft_kv_append_paged_int4(cfg, pool, 2, 16, x, y, _i32([4, 5, 6]), 3, st))
    assert ft.ft_read_device_status(st) == ft.FT_DEV_RANGE


# ---------------------------------------------------------------- attention
@dataclasses.dataclass
class Attn:
    """One problem: a pool of random entries, tables over shuffled pages, garbage behind every request's end."""
    n_q: int
    n_kv: int
    d: int
    ps: int
    qlens: list
    kvlens: list
    had: int = 0
    seed: int = 0
    pad: int = 0           # extra heads between q rows (strided views)
    spread: float = 1.0    # size of q
    vscale: float = 1.0

    def __post_init__(self):
        g = np.random.default_rng(self.seed + 17 * self.d + self.ps)
        self.cfg = _cfg(self.n_q, self.n_kv, self.d, self.had)
        self.B, self.total = len(self.qlens), int(sum(self.qlens))
        self.cu = np.concatenate([[0], np.cumsum(self.qlens)])
        need = [-(-k // self.ps) for k in self.kvlens]
        self.n_pages = sum(need) + 2
        ids = g.permutation(self.n_pages)
        self.table = np.full((self.B, max(max(need), 1) + 1), -5)
        blocks = self.n_pages * self.n_kv
        half = g.integers(0, 1 << 16, (blocks, self.ps * self.d // 2), dtype=np.uint16)
        sc = np.exp(g.normal(-1, 0.5, (blocks, self.ps, 2))).astype(np.float32)
        sc[..., 1] *= self.vscale
        if blocks * self.ps > 40:
            sc[0, 3, 1] = 0.0                              # an entry of V that is zero
            half.reshape(blocks, -1)[0, self.ps * self.d // 4:] &= 0xC0C0  # its page: V codes zero
        bits = synth._to_bf16(sc)[0]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            if self.kvlens[b] % self.ps:                     # NaN and infinity behind the end
                page = ids[at + n - 1]
                tail = bits.reshape(self.n_pages, self.n_kv, self.ps, 2)[page, :, self.kvlens[b] % self.ps:]
                tail[..., 0], tail[..., 1] = 0x7FC0, 0xFF80
            at += n
        raw = np.concatenate([half.view(np.uint8).reshape(blocks, -1), bits.view(np.uint8).reshape(blocks, -1)], 1)
        self.pool_np = raw
        self.pool = torch.from_numpy(raw.reshape(-1)).cuda()
        x, xf = _bf16(g, self.total + 2, self.n_q + self.pad, self.d)
        self.q = (x * self.spread)[:, :self.n_q]
        self.qf = self.q.float().cpu().numpy().astype(np.float64)
        self.scale = self.d ** -0.5

    def set_scales(self, b, positions, k=None, v=None):
        """K and V scales (floats, rounded down to BF16) of request b's positions, in every head."""
        bits = self.pool_np[:, -4 * self.ps:].view(np.uint16).reshape(self.n_pages, self.n_kv, self.ps, 2)
        for pos in positions:
            for i, x in enumerate((k, v)):
                if x is not None:
                    bits[self.table[b, pos // self.ps], :, pos % self.ps, i] = np.float32(x).view(np.uint32) >> 16
        self.pool = torch.from_numpy(self.pool_np.reshape(-1)).cuda()

    def run(self, max_q=None, ws=None, stream=None, o=None, status=None, q=None):
        o = torch.full((self.total + 2, self.n_q, self.d), 7.0, dtype=torch.bfloat16, device="cuda") if o is None else o
        max_q = max(self.qlens) if max_q is None else max_q
        st = _status() if status is None else status
        if ws is None:
            ws = torch.full((ft.ft_attn_paged_workspace_bytes(self.cfg, self.B, self.total, max(max_q, 1)),), 0xFF,
                            dtype=torch.uint8, device="cuda")
        ft.check(ft.ft_attn_paged_int4(self.cfg, self.pool, self.n_pages, self.ps, self.q if q is None else q, _i32(self.cu),
                                       _i32(self.kvlens), _i32(self.table), self.B, self.total, max(max_q, 1), self.scale, o, ws,
                                       st, stream))
        torch.cuda.synchronize()
        return o, int(st.item())

    def check(self, o, reqs=None, heads=None, floor=2.0 ** -35):
        G = self.n_q // self.n_kv
        got = o.float().cpu().numpy().astype(np.float64)
        assert (got[self.total:] == 7.0).all()               # rows behind the last sequence
        k, v, ks, vs = paged.unpack_pages(self.pool_np, self.n_kv, self.ps, self.d)
        worst = 0.0
        for b in range(self.B) if reqs is None else reqs:
            n, kv = self.qlens[b], self.kvlens[b]
            if not n:
                continue
            pages = self.table[b, :-(-kv // self.ps)]
            for h in range(self.n_q) if heads is None else heads:
                j = h // G
                kh, vh = (c[pages, j].reshape(-1, self.d)[:kv] * s[pages, j].reshape(-1, 1)[:kv] for c, s in ((k, ks), (v, vs)))
                rows = slice(self.cu[b], self.cu[b] + n)
                o64, vn, dn = paged.attend_rows(self.qf[rows, h], kh, vh, self.had or self.d, self.scale, kv - n)
                err = np.linalg.norm(got[rows, h] - o64, axis=-1)
                tol = (2.0 ** -10 * dn + 2.0 ** -11 + 2.0 ** -16) * vn + 2.0 ** -8 * np.linalg.norm(o64, axis=-1)
                tol += kv * floor * vs[pages, j].reshape(-1)[:kv].max(initial=0.0) * 7 * self.d ** 0.5
                empty = vn == 0
                assert not got[rows, h][empty].any()
                assert np.all(err <= tol), (b, h, float(np.max(err / np.maximum(tol, 1e-300))))
                worst = max(worst, float(np.max(err / np.maximum(tol, 1e-300))))
        return worst


def _case(*args, **more):
    return args, more


ATTN = [
    # single tokens: one, a tile's edges, pages of each size, ragged, requests without rows
    _case(8, 2, 64, 16, [1], [1]), _case(32, 8, 128, 64, [1], [1025]), _case(8, 8, 128, 16, [1, 1, 1], [15, 16, 17]),
    _case(32, 8, 128, 128, [1] * 5, [127, 128, 129, 1, 700]), _case(64, 8, 128, 32, [1, 0, 1], [333, 64, 2]),
    _case(42, 6, 64, 64, [1] * 9, [5, 63, 64, 65, 1, 400, 128, 31, 33], pad=12),
    _case(12, 4, 128, 16, [1, 1], [4000, 3], had=32), _case(4, 4, 64, 128, [1], [513], had=1),
    # drafts of a few tokens
    _case(32, 8, 128, 64, [2, 5, 1], [2, 700, 64]), _case(64, 8, 128, 16, [4, 3], [68, 1000], pad=16), _case(8, 2, 64, 32, [7, 8], [7, 90]),
    # prompts and chunks: row and key tiles' edges, no history, long history, odd groups
    _case(8, 2, 64, 16, [33, 1, 65, 130], [33, 50, 65, 1000]), _case(32, 8, 128, 64, [64, 63, 65], [64, 127, 300]),
    _case(16, 2, 128, 32, [129, 0, 17], [129, 10, 400]), _case(6, 2, 128, 128, [100, 200], [357, 200]),
    _case(4, 4, 128, 16, [300, 128], [300, 256]), _case(42, 6, 64, 64, [90, 40], [217, 40], pad=2), _case(7, 1, 128, 64, [259], [640]),
    _case(64, 8, 128, 64, [48, 80], [1500, 80], had=64),
    # tokens before position 0 see nothing; a request whose cache is empty
    _case(8, 2, 64, 16, [5, 3, 1], [2, 0, 0]), _case(8, 2, 128, 64, [150, 90], [70, 0]), _case(32, 8, 128, 64, [1, 1], [0, 9]),
    # sharp softmaxes, tiny and huge V scales
    _case(8, 2, 128, 64, [40], [500], spread=16.0), _case(8, 2, 64, 16, [1, 1], [300, 77], spread=16.0),
    _case(8, 2, 128, 64, [1, 70], [300, 300], vscale=1e20), _case(8, 2, 64, 64, [1, 70], [300, 300], vscale=1e-20),
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention(i):
    a = Attn(*ATTN[i][0], **ATTN[i][1])
    o, st = a.run()
    assert st == 0
    a.check(o)
    o2, _ = a.run()
    assert torch.equal(o, o2)                                 # the same bits again


@pytest.mark.parametrize("qlens,kvlens,n_q", [([1] * 3, [9000, 33000, 40], 32), ([70], [20000], 64), ([1200, 33], [1200, 9000], 32),
                                              ([600, 1, 2], [5000, 6000, 2], 16)])
def test_attention_long(qlens, kvlens, n_q):
    a = Attn(n_q, 8, 128, 64, qlens, kvlens)
    o, st = a.run()
    assert st == 0
    a.check(o, heads=[0, n_q // 2 + 1, n_q - 1])


def test_attention_max_q_is_a_bound_only():
    a = Attn(32, 8, 128, 64, [1, 3, 40], [100, 300, 200])
    for m in (40, 41, 1000):
        o, st = a.run(max_q=m)
        assert st == 0
        a.check(o)


def test_attention_over_q_in_place():
    a = Attn(32, 8, 128, 64, [1, 30, 2], [100, 300, 2])
    want, _ = a.run()
    buf = a.q.clone()
    o, st = a.run(o=buf, q=buf)
    assert st == 0 and torch.equal(o[:a.total], want[:a.total])


@pytest.mark.parametrize("qlens", [[1, 1, 1], [40, 2, 60]])
def test_attention_bad_requests(qlens):
    """Device-side conditions: each flags, spoils only its own request, and the call completes."""
    a = Attn(8, 2, 128, 16, qlens, [50, 70, 90])
    want, _ = a.run()
    a.table[1, 2] = a.n_pages                                 # outside the pool
    o, st = a.run()
    assert st == ft.FT_DEV_RANGE
    a.check(o, reqs=[0, 2])
    a.table[1, 2] = 0
    a.kvlens[1] = a.table.shape[1] * 16 + 1                     # more pages than the table has
    o, st = a.run()
    assert st == ft.FT_DEV_CAPACITY and not o[a.cu[1]:a.cu[2]].any()
    a.check(o, reqs=[0, 2])
    a.kvlens[1] = -4
    o, st = a.run()
    assert st == ft.FT_DEV_CAPACITY and not o[a.cu[1]:a.cu[2]].any()
    a.kvlens[1] = 70
    cu = a.cu.copy()
    a.cu = np.array([0, cu[1], cu[1] - 1, cu[1] - 1])            # descending
    o, st = a.run()
    assert st == ft.FT_DEV_RANGE and torch.equal(o[:cu[1]], want[:cu[1]]) and (o[cu[1]:] == 7.0).all()
    a.cu = np.array([0, cu[1], cu[2], a.total + 1])              # past the rows of q
    o, st = a.run(max_q=max(qlens) + 1)
    assert st == ft.FT_DEV_RANGE and (o[cu[2]:] == 7.0).all()
    a.cu = cu
    if max(qlens) > 1:
        o, st = a.run(max_q=50)                                 # request 2 has more rows
        assert st == ft.FT_DEV_RANGE and (o[cu[2]:] == 7.0).all()
        a.check(torch.where((torch.arange(a.total + 2, device="cuda") < cu[2])[:, None, None], o, 7.0), reqs=[0, 1])


@pytest.mark.parametrize("n", [1, 33])
def test_attention_bad_query(n):
    """A NaN or an oversized query flags and spoils only its own row and head."""
    a = Attn(8, 2, 128, 64, [n, n], [200, 100])
    want, _ = a.run()
    q = a.q.clone()
    q[0, 3, 7] = float("nan")
    q[n, 5, 2] = 1e30
    o, st = a.run(q=q)
    assert st == ft.FT_DEV_RANGE and torch.isnan(o[0, 3].float()).all()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[0, 3], keep[n, 5] = False, False
    a.check(torch.where(keep, o, want))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 2.0 ** 9, 2.0 ** 13])
@pytest.mark.parametrize("n,d", [(5, 128), (200, 128), (200, 64)])
def test_attention_later_entries_do_not_reach_earlier_rows(n, d, what):
    """An entry of the new tokens' own with scales that are not finite, or far above its neighbours', is not there for
    the tokens before it (its neighbours in the same tile keep all their digits)."""
    a = Attn(32, 8, d, 64, [n, n], [n + 60, n + 60])
    first = n // 2                                             # tokens before the entry
    a.set_scales(0, [60 + first], k=what, v=what)
    o, _ = a.run()
    a.check(o, reqs=[1])
    # request 0 as if it ended before the entry
    a.qlens, a.kvlens, a.total, a.cu = [first, 0], [60 + first, 0], first, np.array([0, first, first])
    tail = torch.full_like(o[:2], 7.0)
    a.check(torch.cat([o[:first], tail]), reqs=[0], floor=2.0 ** -27)


@pytest.mark.parametrize("big", [2.0 ** 60, 1.0, 2.0 ** -60])
@pytest.mark.parametrize("n", [1, 70])
def test_attention_entries_without_values_keep_their_weight(n, big):
    """Entries whose V is zero (scale 0) take their part of the softmax, however large or small the others' values are."""
    a = Attn(8, 2, 128, 64, [n], [70])
    a.set_scales(0, range(32), v=0.0)                          # whole groups and tiles of them
    a.set_scales(0, range(32, 70), v=big)
    a.set_scales(0, [40, 69], v=0.0)
    o, st = a.run()
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("n", [1, 150])
def test_attention_scales_of_many_sizes(n):
    """Neighbouring scales that differ by up to 2^15: exact products still."""
    a = Attn(8, 2, 128, 64, [n], [400])
    g = np.random.default_rng(3)
    for pos in range(400):
        a.set_scales(0, [pos], k=2.0 ** -g.integers(0, 15), v=2.0 ** -g.integers(0, 15))
    o, st = a.run()
    assert st == 0
    a.check(o, floor=2.0 ** -27)     # operands 2^8 larger, so weights of FP16's smallest step 2^-24 count 2^8 times as much


@pytest.mark.parametrize("B,n_q,n_kv,d,ps,new,top", [(150, 4, 2, 64, 16, 1, 90), (1100, 2, 1, 64, 16, 1, 40), (40, 8, 2, 128, 64, 20, 200),
                                                     (600, 2, 2, 64, 32, 9, 60)])
def test_attention_of_many_requests(B, n_q, n_kv, d, ps, new, top):
    """More requests than lanes, threads and search steps, some without rows or without a cache."""
    g = np.random.default_rng(B)
    q = g.integers(0, new + 1, B)
    q[g.integers(0, B, 3)] = new
    if new > 1:
        q[7] = 33                                              # (a group's rows pass 32: the kernel for many rows)
    kv = q + g.integers(0, top, B)
    kv[g.integers(0, B, 3)] = 0
    a = Attn(n_q, n_kv, d, ps, [int(x) for x in q], [int(x) for x in kv])
    o, st = a.run()
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("had", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("n,d", [(1, 128), (40, 128), (40, 64)])
def test_attention_rotations_of_every_size(n, d, had):
    a = Attn(8, 2, d, 32, [n, 1], [n + 77, 130], had=had)
    o, st = a.run()
    assert st == 0
    a.check(o)


@pytest.mark.parametrize("qlens,kvlens", [([1, 1], [700, 33]), ([3, 1], [260, 1])])
def test_attention_groups_past_the_librarys_limit_are_refused(qlens, kvlens):
    """64 query heads of one KV head: no configuration of this library (at most eight)."""
    a = Attn(64, 1, 128, 64, qlens, kvlens)
    with pytest.raises(ft.FTError):
        a.run(ws=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))
    assert ft.ft_attn_paged_workspace_bytes(a.cfg, 2, a.total, max(qlens)) == 0


@pytest.mark.parametrize("qlens", [[1, 2, 1], [90, 2, 40]])
@pytest.mark.parametrize("off", [1, 4])
def test_attention_rows_at_odd_addresses(qlens, off):
    """Rows of q and o that start at no 16-byte boundary, and leave gaps that stay as they were."""
    a = Attn(8, 2, 128, 16, qlens, [100, 50, 333])
    want, _ = a.run()
    row = 8 * 128 + 3
    qb, ob = (torch.full((off + (a.total + 2) * row,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    view = lambda t: torch.as_strided(t, (a.total + 2, 8, 128), (row, 128, 1), off)  # noqa: E731
    view(qb).copy_(a.q)
    o, st = a.run(q=view(qb), o=view(ob))
    assert st == 0 and torch.equal(o[:a.total], want[:a.total])
    view(ob)[:a.total] = 7.0
    assert (ob == 7.0).all()


def test_attention_in_parts_over_q_in_place():
    """Rows over a long cache, in parts that a second kernel joins, beside short requests, written over q."""
    a = Attn(16, 2, 128, 64, [40, 3, 0, 17], [5000, 3, 70, 40])
    want, st = a.run()
    assert st == 0
    a.check(want, heads=[0, 9, 15])
    buf = a.q.clone()
    o, st = a.run(o=buf, q=buf)
    assert st == 0 and torch.equal(o[:a.total], want[:a.total])


@pytest.mark.parametrize("qlens,kvlens", [([1] * 6, [3000, 1, 64, 65, 700, 0]), ([150, 1, 40], [150, 2000, 900]), ([40], [6000])])
def test_attention_captured_and_replayed(qlens, kvlens):
    """One capture; the lengths, tables and queries that it reads change on the device between the replays."""
    a = Attn(32, 8, 128, 64, qlens, kvlens)
    want, _ = a.run()
    cu, kv, table, st = _i32(a.cu), _i32(a.kvlens), _i32(a.table), _status()
    q = a.q.clone()
    o = torch.full((a.total + 2, a.n_q, a.d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ft.ft_attn_paged_workspace_bytes(a.cfg, a.B, a.total, max(qlens)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.check(ft.ft_attn_paged_int4(a.cfg, a.pool, a.n_pages, a.ps, q, cu, kv, table, a.B, a.total, max(qlens), a.scale, o, ws,
                                       st))
    for _ in range(2):
        ws.fill_(0xFF)
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    short = [max(x // 2, min(x, 1)) for x in kvlens]
    kv.copy_(_i32(short))
    q.copy_(a.q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    a.kvlens = short
    again, _ = a.run(q=q)
    assert torch.equal(o, again) and st.item() == 0


def test_attention_offsets_past_32_bits():
    """Pages behind the first 4 GiB (and 2^32 bytes of one head's stride) are addressed with 64 bits."""
    cfg, ps, d, h = _cfg(8, 8, 128), 64, 128, 8
    n_pages = (5 << 30) // (h * ps * (d + 4))
    pool = torch.zeros(ft.ft_kv_pages_bytes(cfg, n_pages, ps), dtype=torch.uint8, device="cuda")
    g = np.random.default_rng(5)
    n = 150
    x, _ = _bf16(g, n, 24, d)
    pages = np.array([n_pages - 1, 3, n_pages - 2])
    slots = pages[np.arange(n) // ps] * ps + np.arange(n) % ps
    small = torch.zeros(ft.ft_kv_pages_bytes(cfg, 3, ps), dtype=torch.uint8, device="cuda")
    res = []
    for buf, np_, sl, table in ((pool, n_pages, slots, pages), (small, 3, np.arange(n), np.arange(3))):
        st = _status()
        ft.check(ft.ft_kv_append_paged_int4(cfg, buf, np_, ps, x[:, 8:16], x[:, 16:], _i32(sl), n, st))
        ko, vo = (torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ft.check(ft.ft_kv_read_paged_int4(cfg, buf, np_, ps, _i32(sl), n, ko, vo, st))
        for qn in (1, n):
            o = torch.empty((qn, h, d), dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(ft.ft_attn_paged_workspace_bytes(cfg, 1, qn, qn), dtype=torch.uint8, device="cuda")
            ft.check(ft.ft_attn_paged_int4(cfg, buf, np_, ps, x[:qn, :8], _i32([0, qn]), _i32([n]), _i32([table]), 1, qn, qn,
                                           d ** -0.5, o, ws, st))
            res.append(o)
        res += [ko, vo]
        assert ft.ft_read_device_status(st) == 0
    for p, q in zip(res[:4], res[4:]):
        assert torch.equal(p, q)


# ---------------------------------------------------------------- log probabilities
def test_lengths_next_to_2_to_31_are_not_served():
    a = Attn(2, 1, 64, 128, [1], [10])
    table = torch.zeros((1, 1 << 24), dtype=torch.int32, device="cuda")
    st, o = _status(), torch.full((1, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for rows in (1, 40):
        ws = torch.empty(ft.ft_attn_paged_workspace_bytes(a.cfg, 1, rows, rows), dtype=torch.uint8, device="cuda")
        q = a.q[:1].expand(rows, 2, 64).contiguous()
        o = torch.full_like(q, 7.0)
        ft.check(ft.ft_attn_paged_int4(a.cfg, a.pool, a.n_pages, 128, q, _i32([0, rows]), _i32([2 ** 31 - 250]), table, 1, rows, rows,
                                       0.1, o, ws, st))
        assert ft.ft_read_device_status(st) == ft.FT_DEV_CAPACITY and not o.any()
    st, kv, cu, slots = _status(), _i32([7]), _i32([7, 7]), _i32([7] * 5)
    ft.check(ft.ft_kv_page_map(128, a.n_pages, _i32([2 ** 31 - 2]), _i32([5]), 1, table, _i32([0, 1]), _i32([0]), None, cu, kv, slots, st))
    assert ft.ft_read_device_status(st) == ft.FT_DEV_CAPACITY
    assert kv.tolist() == [0] and slots.tolist() == [-1] * 5 and cu.tolist() == [0, 5] and not table.any()


def _logprobs(x, t, top, want_all=True):
    n = x.shape[0]
    f = lambda *s: torch.full(s, 5.0, dtype=torch.float32, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, 5, dtype=torch.int32, device="cuda")  # noqa: E731
    out = {"logprob": f(n), "entropy": f(n), "rank": i(n), "top_ids": i(n, max(top, 1)), "top_logprobs": f(n, max(top, 1))}
    st = _status()
    ft.check(ft.ft_logprobs(x, None if t is None else _i32(t), *(out[k] if want_all else None for k in out), top, st))
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}, int(st.item())


def _check_logprobs(x, t, top):
    got, st = _logprobs(x, t, top)
    assert st == 0
    want = paged.logprobs(x.double().cpu().numpy(), t, top)
    with np.errstate(over="ignore"):                           # what FP32 cannot hold is its infinity
        want = {k: v.astype(np.float32).astype(np.float64) if v.dtype == np.float64 else v for k, v in want.items()}
    V = x.shape[1]
    rel = (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -21          # of the sum z, and of its logarithm absolutely
    xa = np.abs(x.float().cpu().numpy())
    xa = np.where(np.isfinite(xa), xa, 0).max(-1)
    tol = rel + 2.0 ** -22 * (xa + np.log(V) + 1)
    np.testing.assert_array_equal(got["rank"], want["rank"])
    fin = np.isfinite(want["logprob"])
    np.testing.assert_array_equal(got["logprob"][~fin], want["logprob"][~fin])
    assert np.all(np.abs(got["logprob"][fin] - want["logprob"][fin]) <= tol[fin])
    # entropy = log z + sum e d / z: the second sum's terms add up to at most entropy + log V
    assert np.all(np.abs(got["entropy"] - want["entropy"]) <= rel + 2 * rel * (want["entropy"] + np.log(V)) + 2.0 ** -22 * np.log(V))
    if top:
        np.testing.assert_array_equal(got["top_ids"], want["top_ids"])
        fin = np.isfinite(want["top_logprobs"])
        np.testing.assert_array_equal(got["top_logprobs"][~fin], want["top_logprobs"][~fin])
        err = np.abs(np.where(fin, got["top_logprobs"], 0) - np.where(fin, want["top_logprobs"], 0))
        assert np.all(err <= tol[:, None])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top,pad", [(1, 1, 1, 0), (1, 128256, 5, 0), (3, 37, 32, 1), (32, 50257, 20, 47), (5, 1000, 0, 3),
                                         (40, 4096, 1, 0), (700, 513, 8, 0), (2, 200003, 32, 5), (17, 32000, 3, 7)])
def test_logprobs(N, V, top, pad, dtype):
    g = np.random.default_rng(N + V)
    x = torch.from_numpy((g.normal(0, 3, (N, V + pad))).astype(np.float32)).to(dtype).cuda()[:, :V]
    t = g.integers(0, V, N)
    t[0], t[-1] = 0, V - 1
    _check_logprobs(x, t, top)


@pytest.mark.parametrize("V", [50, 20000])
def test_logprobs_ties_masks_and_order(V):
    """Equal logits, masked vocabularies, sorted rows either way, a single survivor, huge and tiny values."""
    top = 16
    x = torch.zeros((9, V))
    x[1] = -float("inf")
    x[1, 3::7] = 1.0                                        # masked, the rest tied
    x[2] = torch.arange(V).float() / V
    x[3] = -torch.arange(V).float() / V
    x[4] = -float("inf")
    x[4, V // 2] = -3e38                                      # one survivor
    x[5] = -3.3e38
    x[5, 4] = 3.3e38                                         # a span beyond FP32's range
    x[6] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)     # zeros of both signs are equal
    x[7] = 1e-40
    x[7, 9] = 2e-40                                           # subnormal
    x[8] = torch.randint(0, 4, (V,), generator=torch.Generator().manual_seed(1)).float()
    t = np.array([V - 1, 3, 0, V - 1, V // 2, 4, 7, 9, V // 3])
    _check_logprobs(x.cuda(), t, top)
    t[1], t[4] = 4, 0                                         # masked targets: -infinity, behind every survivor
    _check_logprobs(x.cuda(), t, top)


def test_logprobs_conditions():
    x = torch.randn((6, 300), generator=torch.Generator().manual_seed(2)).cuda()
    t = [5, -1, 300, -2, 7, 8]
    got, st = _logprobs(x, t, 2)
    assert st == ft.FT_DEV_RANGE
    assert got["logprob"][1] == 0 and got["rank"][1] == -1
    assert np.isnan(got["logprob"][[2, 3]]).all() and (got["rank"][[2, 3]] == -1).all()
    assert np.isfinite(got["entropy"]).all() and (got["top_ids"] >= 0).all()
    got, st = _logprobs(x, [5, -1, 0, 1, 2, 3], 2)
    assert st == 0
    y = x.clone()
    y[0, 290], y[1, 3], y[2] = float("nan"), float("inf"), -float("inf")
    got, st = _logprobs(y, [1, 2, 3, 4, 5, 6], 2)
    assert st == ft.FT_DEV_RANGE
    for k in ("logprob", "entropy"):
        assert np.isnan(got[k][:3]).all() and np.isfinite(got[k][3:]).all()
    assert np.isnan(got["top_logprobs"][:3]).all() and (got["top_ids"][:3] == -1).all() and (got["rank"][:3] == -1).all()
    got, st = _logprobs(x, None, 0, want_all=False)              # nothing asked for
    assert st == 0 and (got["logprob"] == 5).all()


# ---------------------------------------------------------------- together
class Server:
    """A serving loop's device state: one layer's attention as a model would call it, greedy tokens from the logits."""

    def __init__(self, B, ps=16, n_pages=64, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.B, self.ps, self.n_pages, self.V = B, ps, n_pages, 1000
        self.cfg = ft.make_cfg(1024, 8, 2, 128, 512)
        r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        self.wqkv, self.emb = r(1024, 12 * 128) / 32, r(self.V, 1024)
        self.lm, self.gamma = r(self.V, 1024).to(torch.bfloat16) / 8, torch.ones(1024, device="cuda")
        self.pool = torch.full((ft.ft_kv_pages_bytes(self.cfg, n_pages, ps),), 0xFF, dtype=torch.uint8, device="cuda")
        self.table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.head, self.ctx, self.cu, self.status = z(1), z(B), z(B + 1), z(1)
        self.one, self.tokens, self.logits = z(B) + 1, z(B, 1), torch.zeros((B, self.V), device="cuda")
        self.lp, self.top = torch.zeros(B, device="cuda"), torch.zeros((B, 1), device="cuda")

    def forward(self, new, tokens, max_q):
        """Appends `tokens` (packed) and returns the attention output of every row."""
        total = tokens.numel()
        slots = torch.empty(total, dtype=torch.int32, device="cuda")
        ft.check(ft.ft_kv_page_map(self.ps, self.n_pages, self.ctx, new, self.B, self.table, self.free, self.head, self.head,
                                   self.cu, self.ctx, slots, self.status))
        x = (self.emb[tokens.view(-1).long()] @ self.wqkv).to(torch.bfloat16).view(total, 12, 128)
        ft.check(ft.ft_kv_append_paged_int4(self.cfg, self.pool, self.n_pages, self.ps, x[:, 8:10], x[:, 10:], slots, total,
                                            self.status))
        o = torch.empty((total, 8, 128), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(ft.ft_attn_paged_workspace_bytes(self.cfg, self.B, total, max_q), dtype=torch.uint8, device="cuda")
        ft.check(ft.ft_attn_paged_int4(self.cfg, self.pool, self.n_pages, self.ps, x[:, :8], self.cu, self.ctx, self.table, self.B,
                                       total, max_q, 128 ** -0.5, o, ws, self.status))
        return o

    def choose(self, h):
        """Greedy token and its log probability from the last rows' states [B, 1024]."""
        ft.check(ft.ft_lm_head_bf16(h, self.gamma, self.lm, self.logits, self.B, self.V, 1024, 1e-5))
        ft.check(ft.ft_logprobs(self.logits, None, None, None, None, self.tokens, self.top, 1, self.status))
        ft.check(ft.ft_logprobs(self.logits, self.tokens.view(-1), self.lp, None, None, None, None, 0, self.status))

    def step(self):
        self.choose(self.forward(self.one, self.tokens, 1).view(self.B, 1024).float())


def test_generation_loop_matches_whole_prompts():
    """Prompts, then decode steps (captured once and replayed on another stream): the states equal those of one call over
    all tokens at once, the lengths and pages advance on the device, and tokens and log probabilities agree."""
    B, lens = 3, [20, 1, 33]
    s = Server(B)
    g = torch.Generator().manual_seed(4)
    prompt = torch.randint(0, s.V, (sum(lens),), generator=g).to(torch.int32).cuda()
    o = s.forward(_i32(lens), prompt, max(lens))
    last = torch.tensor(np.cumsum(lens) - 1).cuda()
    s.choose(o[last].view(B, 1024).float())
    chosen, lps = [s.tokens.clone()], [s.lp.clone()]
    s.step()
    torch.cuda.synchronize()
    chosen.append(s.tokens.clone())
    lps.append(s.lp.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    keep = {k: v.clone() for k, v in vars(s).items() if isinstance(v, torch.Tensor)}
    with torch.cuda.graph(graph, stream=side):
        s.step()
    for k, v in keep.items():
        assert torch.equal(v, getattr(s, k)), k               # capturing ran nothing
    for _ in range(30):
        graph.replay()
        chosen.append(s.tokens.clone())
        lps.append(s.lp.clone())
    torch.cuda.synchronize()
    steps = len(chosen) - 1
    assert s.status.item() == 0
    assert s.ctx.tolist() == [n + steps for n in lens]
    assert s.head.item() == sum(-(-(n + steps) // s.ps) for n in lens)
    # all tokens again in one call, on a fresh pool
    w = Server(B)
    seq = torch.stack(chosen)[..., 0]                          # [steps + 1, B]
    packed, first = [], 0
    for b, n in enumerate(lens):
        packed += [prompt[first:first + n], seq[:steps, b]]
        first += n
    total = [n + steps for n in lens]
    o = w.forward(_i32(total), torch.cat(packed), max(total))
    last = torch.tensor(np.cumsum(total) - 1).cuda()
    w.choose(o[last].view(B, 1024).float())
    assert w.status.item() == 0
    # the two ways sum in another order: BF16 outputs a step apart move a logit by under 1e-2 here
    assert (w.lp - lps[-1]).abs().max() < 0.1
    logits = w.logits.gather(1, chosen[-1].long())
    assert (w.logits.max(-1, keepdim=True).values - logits).max() < 0.1


def test_two_streams_with_their_own_workspaces():
    a, b = Attn(32, 8, 128, 64, [1] * 8, [4000] * 8), Attn(32, 8, 128, 64, [300], [2000])
    wa, wb = a.run()[0], b.run()[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        outs = []
        for x, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                o = torch.full((x.total + 2, x.n_q, x.d), 7.0, dtype=torch.bfloat16, device="cuda")
                ws = torch.empty(ft.ft_attn_paged_workspace_bytes(x.cfg, x.B, x.total, max(x.qlens)), dtype=torch.uint8,
                                 device="cuda")
                args = [_i32(x.cu), _i32(x.kvlens), _i32(x.table)]
                ft.check(ft.ft_attn_paged_int4(x.cfg, x.pool, x.n_pages, x.ps, x.q, *args, x.B, x.total, max(x.qlens), x.scale, o,
                                               ws))
                outs.append((o, ws, args))
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], wa) and torch.equal(outs[1][0], wb)


def test_binding_refuses_what_it_cannot_pass():
    a = Attn(8, 2, 128, 64, [3], [10])
    ws = torch.empty(ft.ft_attn_paged_workspace_bytes(a.cfg, 1, 3, 3), dtype=torch.uint8, device="cuda")
    o = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda q=a.q, kv=_i32([10]), pool=a.pool, out=o: ft.ft_attn_paged_int4(  # noqa: E731
        a.cfg, pool, a.n_pages, 64, q, _i32([0, 3]), kv, _i32(a.table), 1, 3, 3, 0.1, out, ws)
    assert call() == ft.FT_OK
    for bad in (dict(q=a.q.cpu()), dict(q=a.q.float()), dict(q=a.q.half()), dict(out=o.half()), dict(q=a.q.transpose(1, 2)), dict(kv=_i32([10]).long()), dict(q=a.q[:2]),
                dict(pool=a.pool[:-1]), dict(out=o[:, :, ::2]), dict(kv=torch.tensor([10], dtype=torch.int32))):
        with pytest.raises(ValueError):
            call(**bad)
    x = torch.randn((2, 50), device="cuda")
    with pytest.raises(ValueError):
        ft.ft_logprobs(x.half(), _i32([0, 0]), torch.zeros(2, device="cuda"), None, None, None, None, 0)
    with pytest.raises(ValueError):
        ft.ft_logprobs(x[:, ::2], _i32([0, 0]), None, None, _i32([0, 0]), None, None, 0)
    with pytest.raises(ValueError):
        ft.ft_logprobs(x, _i32([0]), torch.zeros(2, device="cuda"), None, None, None, None, 0)
