"""The paged cache and the log probabilities at the ends of their ranges: sizes next to
2^31, entries without finite scales, scales far apart, calls that follow each other with
nothing in between, and arguments of the wrong type.

Tolerances are those of test_paged_gpu.py (derived there); anything else is exact.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
import int4_weight_kv_gb300 as ft
from int4_weight_kv_gb300 import runtime as rt
from oracle import paged
from tests import gpu_harness as H
from tests.test_paged_gpu import Attn, Server, _bf16, _cfg, _gpu, _i32, _status  # noqa: F401 (_gpu: a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- page map
@pytest.mark.parametrize("alias", [False, True])
def test_page_map_slots_up_to_2_to_31(alias):
    """The slots behind the last row are -1 up to the largest slot map; nothing before it is touched."""
    n, dev = 2 ** 31 - 1, "cuda"
    buf = torch.full((n + 8192,), 77, dtype=torch.int32, device=dev)
    slots = buf[8192:]
    c, t, h, st, cu = _i32([30, 3]), _i32([[5, 6], [4, 4]]), _i32([0]), _status(), _i32([0] * 3)
    kv, ho = (c, h) if alias else (_i32([0, 0]), _i32([0]))
    ft.check(ft.ft_kv_page_map(16, 10, c, _i32([2, 4]), 2, t, _i32([9]), h, ho, cu, kv, slots, st))
    assert ft.ft_read_device_status(st) == 0
    assert cu.tolist() == [0, 2, 6] and kv.tolist() == [32, 7] and ho.tolist() == [0]
    assert slots[:6].tolist() == [6 * 16 + 14, 6 * 16 + 15, 67, 68, 69, 70]
    assert (buf[:8192] == 77).all()
    for a in range(6, n, 1 << 28):
        assert (slots[a:a + (1 << 28)] == -1).all()


def test_page_map_takes_up_to_2_to_31_pages():
    """Sixteen requests that fill their table rows from a free list of 2^31 - 1 entries."""
    per, dev = 1 << 27, "cuda"
    n_pages, n_free = (2 ** 31 - 1) // 16, 2 ** 31 - 1
    free = torch.empty(n_free, dtype=torch.int32, device=dev)
    for a in range(0, n_free, 1 << 28):
        b = min(a + (1 << 28), n_free)
        free[a:b] = (torch.arange(a, b, device=dev) % n_pages).to(torch.int32)
    table = torch.full((16, per), -1, dtype=torch.int32, device=dev)
    new = [2 ** 31 - 1] * 15 + [(per - 1) * 16]
    kv, cu, ho, st, slots = _i32([0] * 16), _i32([0] * 17), _i32([0]), _status(), _i32([7] * 5)
    ft.check(ft.ft_kv_page_map(16, n_pages, _i32([0] * 16), _i32(new), 16, table, free, None, ho, cu, kv, slots, st))
    assert ft.ft_read_device_status(st) == ft.FT_DEV_RANGE      # more rows than slots
    assert ho.tolist() == [n_free] and slots.tolist() == [0, 1, 2, 3, 4]
    flat = table.view(-1)
    assert flat[-1].item() == -1
    for a in range(0, n_free, 1 << 28):
        b = min(a + (1 << 28), n_free)
        assert torch.equal(flat[a:b], free[a:b])


@pytest.mark.parametrize("alias", [False, True])
def test_lengths_of_more_rows_than_2_to_31(alias):
    """kv_len is ctx_len + new_len also where the prefix sums end at 2^31 - 1."""
    ctx, new = [5, 100, 0, 7], [2 ** 30] * 3 + [0]
    width = 2 ** 23 + 1
    free = torch.zeros(3 * width, dtype=torch.int32, device="cuda")
    table = torch.zeros((4, width), dtype=torch.int32, device="cuda")
    c, cu, st = _i32(ctx), _i32([0] * 5), _status()
    kv = c if alias else _i32([0] * 4)
    ft.check(ft.ft_kv_page_map(128, 3, c, _i32(new), 4, table, free, None, None, cu, kv, _i32([7] * 5), st))
    assert ft.ft_read_device_status(st) == ft.FT_DEV_RANGE
    assert cu.tolist() == [0, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert kv.tolist() == [c + n for c, n in zip(ctx, new)]


def test_page_map_of_every_batch_size_in_a_fresh_process():
    """Batches around the limits of shared memory, the first of them in a process that has launched nothing else."""
    code = """
import torch, int4_weight_kv_gb300 as ft
i = lambda n: torch.zeros(n, dtype=torch.int32, device='cuda')
for B in (4095, 4070, 4083, 4084, 4090, 4096, 4097, 8191, 8192):
    table, slots, kv = i((B, 1)) - 1, i(B), i(B)
    st = i(1)
    free = torch.arange(B, dtype=torch.int32, device='cuda')
    ft.check(ft.ft_kv_page_map(16, B, i(B), i(B) + 1, B, table, free, None, None, i(B + 1), kv, slots, st))
    assert ft.ft_read_device_status(st) == 0
    assert torch.equal(slots, 16 * free) and (kv == 1).all() and torch.equal(table[:, 0], free)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


# ---------------------------------------------------------------- one call behind the other
def _chain(cfg, ps, n_kv, d, rows, V):
    """Three times page map, placement, reading back and log probabilities of what was read, with nothing in between: the same
    pages and the same slot map with other slots and other data each time.  The results of three replays and an eager run."""
    g = torch.Generator("cuda").manual_seed(len(rows) + sum(rows))
    B, total, dev = len(rows), sum(rows), "cuda"
    need = [-(-n // ps) for n in rows]
    n_pages = sum(need)
    pool = torch.zeros(ft.ft_kv_pages_bytes(cfg, n_pages, ps), dtype=torch.uint8, device=dev)
    free = torch.cat([torch.randperm(n_pages, device=dev, generator=g) for _ in range(3)]).to(torch.int32)
    head, ctx0, new = _i32([0]), _i32([0] * B), _i32(rows)
    table, cu, kv = _i32(np.full((B, max(need)), -1)), _i32([0] * (B + 1)), _i32([0] * B)
    slots, st = _i32([0] * total), _status()
    x = [torch.randn((total, 2 * n_kv, d), device=dev, generator=g).to(torch.bfloat16) for _ in range(3)]
    t = _i32([i % V for i in range(total)])
    f = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    bf = lambda: torch.zeros((total, n_kv, d), dtype=torch.bfloat16, device=dev)  # noqa: E731
    out = [[bf(), bf(), f(total), f(total), _i32([0] * total), _i32([[0] * 3] * total), f(total, 3)] for _ in range(3)]

    def steps():
        head.zero_()
        for k in range(3):
            ko, vo, lp, en, rank, ids, tv = out[k]
            ft.check(ft.ft_kv_page_map(ps, n_pages, ctx0, new, B, table, free, head, head, cu, kv, slots, st))
            ft.check(ft.ft_kv_append_paged_int4(cfg, pool, n_pages, ps, x[k][:, :n_kv], x[k][:, n_kv:], slots, total, st))
            ft.check(ft.ft_kv_read_paged_int4(cfg, pool, n_pages, ps, slots, total, ko, vo, st))
            ft.check(ft.ft_logprobs(ko.view(total, V), t, lp, en, rank, ids, tv, 3, st))

    steps()
    torch.cuda.synchronize()
    res = [[y.clone() for s in out for y in s]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(3):
        pool.fill_(0xFF)
        for y in [slots] + [y for s in out for y in s]:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        res.append([y.clone() for s in out for y in s])
    assert st.item() == 0 and head.item() == 3 * n_pages
    return res


@pytest.mark.parametrize("rows,n_kv,d,ps", [([1] * 32, 8, 128, 64), ([1], 2, 64, 16), ([300, 1, 77, 2000], 8, 128, 32),
                                            ([5, 64, 700], 4, 64, 16)])
def test_calls_behind_each_other_with_and_without_overlap(rows, n_kv, d, ps):
    cfg = _cfg(n_kv, n_kv, d)
    was = ft.ft_set_pdl(0)
    try:
        want = _chain(cfg, ps, n_kv, d, rows, n_kv * d)
        ft.ft_set_pdl(1)
        got = _chain(cfg, ps, n_kv, d, rows, n_kv * d)
    finally:
        ft.ft_set_pdl(was)
    for r in want[1:] + got:
        for x, y in zip(want[0], r):
            assert torch.equal(x, y)


@pytest.mark.parametrize("B", [1, 20])
def test_block_stage_behind_a_page_map_that_advances_its_positions(B):
    """The attention stage reads the positions that a page map has just advanced."""
    lay = H.make_layer(synth.TINY, 1)
    pb = H.make_problem(lay, 1, B, 40, max_ctx=64)
    x = torch.from_numpy(pb.x_f32).cuda()
    y, new = torch.empty_like(x), _i32([1] * B)
    table, free = _i32(np.full((B, 8), 0)), _i32(range(8 * B))
    ws, pos, cu, slots, head = rt.alloc_workspace(lay.cfg, B, 64), _i32([0] * B), _i32([0] * (B + 1)), _i32([0] * B), _i32([0])
    lo = ft.ft_decode_workspace_layout(lay.cfg, B, 64)
    n = B * lay.shape.n_q * lay.shape.head_dim
    args = lambda: (lay.cfg, lay.packed, cache, B, 64, x, y, ft.FT_F32, pos, B, ws)  # noqa: E731
    res = []
    for pdl in (0, 1):
        was = ft.ft_set_pdl(pdl)
        try:
            for start in (0, 11, 30):
                cache = pb.cache.clone()
                pos.fill_(start)
                ft.check(ft.ft_decode_block(*args(), None))
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    head.zero_()
                    for _ in range(4):
                        ft.check(ft.ft_kv_page_map(16, 8 * B, pos, new, B, table, free, head, head, cu, pos, slots))
                        ft.check(ft.ft_decode_block_stages(*args(), ft.FT_STAGE_ATTN, None))
                pos.fill_(start)
                graph.replay()
                torch.cuda.synchronize()
                assert pos.tolist() == [start + 4] * B
                res.append((ws[lo.o:lo.o + 2 * n].clone(), cache.clone()))
        finally:
            ft.ft_set_pdl(was)
    for (o0, c0), (o1, c1) in zip(res[:3], res[3:]):
        assert torch.equal(o0, o1) and torch.equal(c0, c1)


# ---------------------------------------------------------------- entries at the ends of their range
BAD = [float("nan"), float("inf")]


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("n,kv,d", [(1, 50, 128), (1, 9000, 128), (4, 70, 64), (8, 300, 128), (200, 260, 128), (200, 260, 64),
                                    (40, 6000, 128)])
def test_rows_that_see_an_entry_without_finite_scales_are_nan(n, kv, d, bad, which):
    """NaN in every channel of the rows at and after the entry, whichever kernel serves them and whichever scale it is; the
    rows before it and the other requests as without it."""
    a = Attn(16, 2, d, 64, [n, n], [kv, kv])
    want, _ = a.run()
    for at in sorted({kv - n + n // 2, kv - 1, kv // 3}):       # among the new tokens, the last, in the history
        keep = a.pool_np.copy()
        a.set_scales(0, [at], **{which: bad})
        o, _ = a.run()
        first = max(0, at - (kv - n))
        assert torch.isnan(o[first:n]).all(), at
        assert torch.equal(o[n:], want[n:])
        a.pool_np[:] = keep
        err = (o[:first].float() - want[:first].float()).norm(dim=-1)
        assert (err <= 2.0 ** -7 * want[:first].float().norm(dim=-1) + 1e-6).all()


@pytest.mark.parametrize("n,kv", [(1, 200), (8, 300), (40, 200), (40, 6000)])
def test_largest_scales(n, kv):
    """Scales up to 2^109 work (keys whose codes are zero: a score of 0 however large the scale); from 2^110 on a row that
    sees them is NaN."""
    a = Attn(16, 2, 128, 64, [n], [kv])
    a.pool_np[:, :64 * 64] = 0                                  # K codes
    a.set_scales(0, range(kv), k=1.0, v=1.0)
    want, st = a.run()
    a.check(want)
    for k, v in ((2.0 ** 109, 1.0), (1.0, 2.0 ** 109)):
        a.set_scales(0, range(kv), k=k, v=v)
        o, st = a.run()
        assert st == 0
        # the same sums but for approximations of log2 and 1 / scale good to 2^-22: at most a BF16 step apart
        ref = want[:n].float() * v
        assert ((o[:n].float() - ref).abs() <= 2.0 ** -7 * ref.abs()).all()
    for k, v in ((2.0 ** 110, 1.0), (2.0 ** 127, 1.0), (1.0, 2.0 ** 110), (1.0, 2.0 ** 127)):
        a.set_scales(0, range(kv), k=1.0, v=1.0)
        a.set_scales(0, [0], k=k, v=v)
        o, st = a.run()
        assert torch.isnan(o[:n]).all()


@pytest.mark.parametrize("up", [30, 104, 110, 118])
@pytest.mark.parametrize("n_kv,d,had", [(8, 128, 0), (2, 64, 0), (2, 128, 1), (2, 64, 16)])
def test_rows_of_every_size_are_read_back(n_kv, d, had, up):
    """Rows around 2^up and 2^-up: as their codes and scales say, rotated back (scales reach 2^118 and 2^-121)."""
    cfg, g = _cfg(n_kv, n_kv, d, had), np.random.default_rng(up)
    x, xf = _bf16(g, 20, 2 * n_kv, d)
    size = torch.tensor([2.0 ** (up if i % 2 else -up) for i in range(20)], device="cuda").view(-1, 1, 1)
    x = (x.float() * size).to(torch.bfloat16)
    pool = torch.zeros(ft.ft_kv_pages_bytes(cfg, 2, 16), dtype=torch.uint8, device="cuda")
    st, sl = _status(), _i32(range(20))
    ft.check(ft.ft_kv_append_paged_int4(cfg, pool, 2, 16, x[:, :n_kv], x[:, n_kv:], sl, 20, st))
    out = [torch.zeros((20, n_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ft.check(ft.ft_kv_read_paged_int4(cfg, pool, 2, 16, sl, 20, *out, st))
    assert ft.ft_read_device_status(st) == 0
    codes = paged.unpack_pages(pool.cpu().numpy(), n_kv, 16, d)
    for c, s, o in ((codes[0], codes[2], out[0]), (codes[1], codes[3], out[1])):
        c, s = c.transpose(0, 2, 1, 3).reshape(32, n_kv, d)[:20], s.transpose(0, 2, 1).reshape(32, n_kv)[:20]
        back = oracle.blockdiag_apply(c * s[..., None], had or d)
        got = o.float().cpu().numpy().astype(np.float64)
        # as in test_append_codes_and_read: FP32 additions (2^-20 of the row's norm), then half a BF16 step; values
        # below FP32's smallest normal number lose up to 2^-126 each
        tol = 2.0 ** -8 * np.abs(back) + 2.0 ** -20 * np.linalg.norm(back, axis=-1, keepdims=True) + d * 2.0 ** -126
        assert np.isfinite(got).all() and np.all(np.abs(got - back) <= tol)


@pytest.mark.parametrize("order", ["small_first", "small_last", "mixed"])
@pytest.mark.parametrize("n,kv", [(1, 70), (1, 9000), (8, 500), (70, 400), (40, 6000)])
def test_v_scales_a_factor_of_2_to_100_apart(n, kv, order):
    """Entries whose values are next to nothing keep their weight, whatever comes first, in one share and across several."""
    a = Attn(16, 2, 128, 64, [n], [kv], spread=3.0)
    g = np.random.default_rng(kv)
    pos = np.arange(kv - n + 1)                                  # (every row sees all of these)
    small = {"small_first": pos < kv // 2, "small_last": pos >= kv // 2, "mixed": g.random(len(pos)) < 0.5}[order]
    a.set_scales(0, range(kv), v=2.0 ** 50)
    a.set_scales(0, pos[small], v=2.0 ** -50)
    o, st = a.run()
    assert st == 0
    # many rows: operands of a group with a wide range of scales are 2^8 larger, and so is FP16's smallest step there
    a.check(o, floor=2.0 ** -27)


@pytest.mark.parametrize("big", [2.0 ** 40, 2.0 ** -70])
@pytest.mark.parametrize("n,kv", [(1, 70), (1, 9000), (70, 400), (40, 6000)])
def test_entries_without_values_beside_the_ends_of_their_range(n, kv, big):
    a = Attn(16, 2, 128, 64, [n], [kv], spread=3.0)
    g = np.random.default_rng(kv)
    a.set_scales(0, range(kv), v=big)
    a.set_scales(0, np.nonzero(g.random(kv) < 0.5)[0], v=0.0)
    o, st = a.run()
    assert st == 0
    # FP16's smallest step of a weight counts from the entries without values, whose scale counts as 2^-60
    a.check(o, floor=2.0 ** -35 * max(1.0, 2.0 ** -60 / big))


@pytest.mark.parametrize("n", [1, 150])
def test_attention_scales_2_to_15_below_their_neighbours(n):
    """The documented end of exact products: a scale 2^-15 beside a 1 in every group of 32, for K and for V."""
    a = Attn(8, 2, 128, 64, [n], [400])
    g = np.random.default_rng(3)
    for pos in range(400):
        a.set_scales(0, [pos], k=2.0 ** -g.integers(0, 16), v=2.0 ** -g.integers(0, 16))
    for pos in range(0, 400, 32):
        a.set_scales(0, [pos], k=1.0, v=2.0 ** -15)
        a.set_scales(0, [min(pos + 5, 399)], k=2.0 ** -15, v=1.0)
    o, st = a.run()
    assert st == 0
    a.check(o, floor=2.0 ** -27)


# ---------------------------------------------------------------- arguments
def test_binding_refuses_other_types_of_the_same_width():
    """FP32 where INT32 is read and the other way round, 16-bit and 8-bit types that are not what their bits are taken for."""
    B, dev = 2, "cuda"
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    f = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    ok = dict(ctx=i(B), new=i(B), table=i(B, 2), free=i(4), head=i(1), out=i(1), cu=i(B + 1), kv=i(B), slots=i(4), st=i(1))
    call = lambda **o: (lambda a: ft.ft_kv_page_map(16, 4, a["ctx"], a["new"], B, a["table"], a["free"], a["head"], a["out"],  # noqa: E731
                                                    a["cu"], a["kv"], a["slots"], a["st"]))(dict(ok, **o))
    assert call() == ft.FT_OK
    for k, v in ok.items():
        with pytest.raises(ValueError):
            call(**{k: v.float()})
    cfg = _cfg(2, 2, 64)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    pool = torch.zeros(ft.ft_kv_pages_bytes(cfg, 2, 16), dtype=torch.uint8, device=dev)
    ok = dict(pool=pool, k=bf(3, 2, 64), v=bf(3, 2, 64), slots=_i32([0, 1, 2]), st=i(1))
    add = lambda **o: (lambda a: ft.ft_kv_append_paged_int4(cfg, a["pool"], 2, 16, a["k"], a["v"], a["slots"], 3, a["st"]))(dict(ok, **o))  # noqa: E731
    read = lambda **o: (lambda a: ft.ft_kv_read_paged_int4(cfg, a["pool"], 2, 16, a["slots"], 3, a["k"], a["v"], a["st"]))(dict(ok, **o))  # noqa: E731
    for c in (add, read):
        assert c() == ft.FT_OK
        assert c(k=ok["k"].view(torch.int16), v=ok["v"].view(torch.int16)) == ft.FT_OK     # BF16 bits
        for bad in (dict(pool=pool.view(torch.float8_e4m3fn)), dict(pool=pool.bool()), dict(k=ok["k"].half()), dict(v=ok["v"].half()),
                    dict(slots=ok["slots"].float()), dict(st=f(1))):
            with pytest.raises(ValueError):
                c(**bad)
    ws = torch.zeros(ft.ft_attn_paged_workspace_bytes(cfg, 1, 3, 3), dtype=torch.uint8, device=dev)
    ok = dict(pool=pool, q=bf(3, 2, 64), o=bf(3, 2, 64), cu=_i32([0, 3]), kv=_i32([3]), table=i(1, 1), st=i(1))
    att = lambda **o: (lambda a: ft.ft_attn_paged_int4(cfg, a["pool"], 2, 16, a["q"], a["cu"], a["kv"], a["table"], 1, 3, 3, 0.1,  # noqa: E731
                                                       a["o"], ws, a["st"]))(dict(ok, **o))
    assert att() == ft.FT_OK
    for bad in (dict(cu=ok["cu"].float()), dict(kv=ok["kv"].float()), dict(table=f(1, 1)), dict(st=f(1)), dict(pool=pool.view(torch.float8_e5m2))):
        with pytest.raises(ValueError):
            att(**bad)
    ok = dict(x=f(2, 50), t=i(2), lp=f(2), en=f(2), rank=i(2), ids=i(2, 2), tv=f(2, 2), st=i(1))
    lps = lambda **o: (lambda a: ft.ft_logprobs(a["x"], a["t"], a["lp"], a["en"], a["rank"], a["ids"], a["tv"], 2, a["st"]))(dict(ok, **o))  # noqa: E731
    assert lps() == ft.FT_OK and lps(x=ok["x"].to(torch.bfloat16)) == ft.FT_OK
    for k, v in ok.items():
        with pytest.raises(ValueError):
            lps(**{k: v.to(torch.int32) if v.dtype == torch.float32 else v.float()})
    assert lps(x=ok["x"].to(torch.bfloat16).view(torch.int16)) == ft.FT_OK


# ---------------------------------------------------------------- together
def test_generation_loop_step_by_step():
    """Every step of a captured generation loop against one call over all tokens: each token's log probability, and that the
    token chosen is the largest logit's.  Both paths differ by the order of FP32 sums, FP16 weights and BF16 outputs."""
    B, lens, steps = 3, [20, 1, 33], 31
    s = Server(B)
    prompt = torch.randint(0, s.V, (sum(lens),), generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    o = s.forward(_i32(lens), prompt, max(lens))
    s.choose(o[torch.tensor(np.cumsum(lens) - 1).cuda()].view(B, 1024).float())
    chosen, lps = [s.tokens.clone()], [s.lp.clone()]
    s.step()
    chosen.append(s.tokens.clone())
    lps.append(s.lp.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(steps - 1):
        graph.replay()
        chosen.append(s.tokens.clone())
        lps.append(s.lp.clone())
    torch.cuda.synchronize()
    assert s.status.item() == 0
    w, seq, got = Server(B), torch.stack(chosen)[..., 0], torch.stack(lps)           # [steps + 1, B]
    packed, rows, first = [], [], 0
    for b, n in enumerate(lens):
        packed += [prompt[first:first + n], seq[:steps, b]]
        rows += range(sum(lens[:b]) + b * steps + n - 1, sum(lens[:b + 1]) + (b + 1) * steps)
        first += n
    total = [n + steps for n in lens]
    h = w.forward(_i32(total), torch.cat(packed), max(total))[torch.tensor(rows).cuda()].view(-1, 1024).float()
    # rows in the order of the requests, steps + 1 of each
    logits = torch.empty((len(rows), w.V), device="cuda")
    for a in range(0, len(rows), 32):
        part = h[a:a + 32].contiguous()
        ft.check(ft.ft_lm_head_bf16(part, w.gamma, w.lm, logits[a:a + 32], part.shape[0], w.V, 1024, 1e-5))
    t, lp = seq.T.reshape(-1).contiguous(), torch.empty(len(rows), device="cuda")
    ft.check(ft.ft_logprobs(logits, t, lp, None, None, None, None, 0, w.status))
    torch.cuda.synchronize()
    assert w.status.item() == 0
    # Before its rounding to BF16 an output differs by under 2^-10 (two times FP16's half step of the weights); a rounding
    # turns that into a whole step, 2^-7 at most, with probability difference / step: variance 2^-17.  The norm passes it on;
    # a logit sums it over a row of norm 32 with weights of 1/8, a log probability is the difference of two such sums.
    bound = 5 * 2 ** 0.5 * 2.0 ** -8.5 * 32 / 8
    err = (lp.view(B, -1).T - got).abs()
    assert err.max() < bound, err.max().item()
    gap = logits.max(-1).values - logits.gather(1, t.view(-1, 1).long())[:, 0]
    assert gap.max() < bound, gap.max().item()
    print("largest difference of a log probability", err.max().item(), "of a logit", gap.max().item())
