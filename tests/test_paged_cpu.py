"""Paged cache and log probabilities without a GPU: the oracle's pins, sizes, and
the refusals of the entry points (every call here returns before a launch)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import paged
import synth

FAKE = 4096  # never dereferenced


@pytest.fixture(scope="module")
def ft():
    from int4_weight_kv_gb300 import build as b
    b.build()
    import int4_weight_kv_gb300 as m
    return m


# ---------------------------------------------------------------- oracle pins
def test_page_map_hand_case():
    # page size 16: request 0 fills its page and needs one more, 1 is new, 2 adds nothing
    r = paged.page_map(16, [15, 0, 5], [2, 3, 0], [[7, -1], [-1, -1], [4, -1]], [9, 8, 6])
    assert r["cu"].tolist() == [0, 2, 5, 5] and r["kv_len"].tolist() == [17, 3, 5]
    assert r["table"].tolist() == [[7, 9], [8, -1], [4, -1]] and r["head"] == 2
    assert r["slots"].tolist() == [7 * 16 + 15, 9 * 16, 8 * 16, 8 * 16 + 1, 8 * 16 + 2] and not r["capacity"]


def test_page_map_short_free_list():
    r = paged.page_map(16, [0, 0, 0], [40, 16, 0], [[-1] * 3] * 3, [1, 2, 3], head=1)
    assert r["kv_len"].tolist() == [0, 0, 0] and r["head"] == 1 and r["capacity"]
    assert (r["slots"] == -1).all() and (r["table"] == -1).all()


def test_unpack_one_value_each():
    """A single word set by hand lands on the channels that the layout names."""
    for d in (64, 128):
        pool = np.zeros((1, 1, 16 * (d + 4)), np.uint8)
        p, g, j = 5, 3, d // 32 - 1
        w = 1 | (2 << 3) | (3 << 8) | (7 << 11) | 0x4000 | 0x40           # 1, -2, 3, -7
        for base in (p * d // 2 + (g // 2) * (d // 8) + 4 * j + 2 * (g % 2),
                     8 * d + 2 * d + (g ^ (2 * 2 if d == 128 else 4)) * (d // 8) + 4 * j + 2):
            pool[0, 0, base], pool[0, 0, base + 1] = w & 255, w >> 8
        pool[0, 0, 16 * d + 4 * p:16 * d + 4 * p + 4] = [0x80, 0x3F, 0x00, 0x40]  # 1.0, 2.0
        k, v, ks, vs = paged.unpack_pages(pool, 1, 16, d)
        want = np.zeros(d, np.int8)
        want[32 * j + g + 8 * np.arange(4)] = [1, -2, 3, -7]
        for x in (k, v):
            np.testing.assert_array_equal(x[0, 0, p], want)
            assert np.count_nonzero(x) == 4
        assert ks[0, 0, p] == 1.0 and vs[0, 0, p] == 2.0


def test_attend_rows_is_attention():
    """Against the dense oracle row by row; a row before position 0 is zero."""
    g = np.random.default_rng(3)
    q, k, v = g.normal(size=(4, 64)), g.normal(size=(9, 64)), g.normal(size=(9, 64))
    o, _, _ = paged.attend_rows(q, k, v, 64, 64 ** -0.5, 5)
    for i in range(4):
        want = oracle.blockdiag_apply(oracle.attend(oracle.blockdiag_apply(q[i], 64), k[:6 + i], v[:6 + i]), 64)
        np.testing.assert_allclose(o[i], want, rtol=1e-12, atol=1e-14)
    assert not paged.attend_rows(q, k, v, 64, 0.1, -2)[0][:2].any()


def test_logprobs_closed_forms():
    x = np.zeros((2, 8))
    x[1, 3:] = -np.inf
    r = paged.logprobs(x, [5, 1], 2)
    np.testing.assert_allclose(r["logprob"], [-np.log(8), -np.log(3)])
    np.testing.assert_allclose(r["entropy"], [np.log(8), np.log(3)])
    assert r["rank"].tolist() == [5, 1] and r["top_ids"].tolist() == [[0, 1], [0, 1]]


# ---------------------------------------------------------------- sizes and refusals
def test_page_bytes(ft):
    c = ft.cfg_from_shape(synth.L8B)
    assert ft.ft_kv_pages_bytes(c, 10, 64) == 10 * 8 * 64 * 132
    assert ft.ft_kv_pages_bytes(ft.cfg_from_shape(synth.TINY), 3, 16) == 3 * 2 * 16 * 68
    assert ft.ft_kv_pages_bytes(c, 1 << 22, 64) == (1 << 22) * 8 * 64 * 132       # 64-bit
    assert ft.ft_kv_pages_bytes(c, 10, 48) == 0 and ft.ft_kv_pages_bytes(c, 0, 64) == 0
    assert ft.ft_kv_pages_bytes(c, 1 << 30, 64) == 0                              # slots past 32 bits


def test_page_map_refusals(ft):
    lib = ft.lib()
    ok = dict(ps=16, pages=8, ctx=FAKE, new=FAKE, B=2, table=FAKE, stride=4, free=FAKE, n_free=3, head=None, out=None,
              cu=FAKE, kv=FAKE, slots=FAKE, n_slots=5)
    call = lambda **o: lib.ft_kv_page_map(*dict(ok, **o).values(), None, None)  # noqa: E731
    assert call(ps=24) == ft.FT_ERR_UNSUPPORTED and call(B=8193) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(ctx=None), dict(new=None), dict(table=None), dict(cu=None), dict(kv=None), dict(B=0), dict(stride=0),
                dict(n_free=-1), dict(free=None), dict(slots=None), dict(n_slots=-1), dict(pages=0)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_append_and_read_refusals(ft):
    lib, c = ft.lib(), ft.cfg_from_shape(synth.L8B)
    ok = dict(pages=FAKE, n=8, ps=64, k=FAKE, ks=1024, v=FAKE, vs=1024, slots=FAKE, total=3)
    call = lambda **o: lib.ft_kv_append_paged_int4(ctypes.byref(c), *dict(ok, **o).values(), None, None)  # noqa: E731
    assert call(total=0) == ft.FT_OK and call(ps=8) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(pages=None), dict(pages=FAKE + 8), dict(n=0), dict(k=None), dict(v=None), dict(slots=None),
                dict(total=-1), dict(ks=1023), dict(vs=0)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad
    ok = dict(pages=FAKE, n=8, ps=64, slots=FAKE, total=3, k=FAKE, v=FAKE)
    call = lambda **o: lib.ft_kv_read_paged_int4(ctypes.byref(c), *dict(ok, **o).values(), None, None)  # noqa: E731
    assert call(total=0) == ft.FT_OK and call(ps=256) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(pages=None), dict(slots=None), dict(k=None), dict(v=None), dict(total=-2)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_attention_refusals(ft):
    lib, c = ft.lib(), ft.cfg_from_shape(synth.L8B)
    size = ft.ft_attn_paged_workspace_bytes(c, 4, 100, 40)
    assert size > 0 and ft.ft_attn_paged_workspace_bytes(c, 0, 100, 40) == 0
    assert ft.ft_attn_paged_workspace_bytes(c, 4, 100, 0) == 0
    ok = dict(pages=FAKE, n=8, ps=64, q=FAKE, qs=4096, cu=FAKE, kv=FAKE, table=FAKE, stride=4, B=4, total=100, max_q=40,
              scale=0.1, o=FAKE, os=4096, ws=FAKE, wsb=size)
    call = lambda **o: lib.ft_attn_paged_int4(ctypes.byref(c), *dict(ok, **o).values(), None, None)  # noqa: E731
    assert call(total=0) == ft.FT_OK and call(wsb=size - 1) == ft.FT_ERR_WORKSPACE
    assert call(ps=40) == ft.FT_ERR_UNSUPPORTED
    for big in (dict(total=2 ** 29), dict(stride=2 ** 28), dict(B=8193)):
        assert call(wsb=2 ** 60, **big) == ft.FT_ERR_UNSUPPORTED, big
    for bad in (dict(pages=None), dict(q=None), dict(o=None), dict(cu=None), dict(kv=None), dict(table=None), dict(ws=None),
                dict(ws=FAKE + 4), dict(B=0), dict(total=-1), dict(max_q=0), dict(stride=0), dict(qs=4095), dict(os=1),
                dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_logprobs_refusals(ft):
    lib = ft.lib()
    ok = dict(x=FAKE, dt=ft.FT_F32, stride=100, N=2, V=100, t=FAKE, top=4, lp=FAKE, en=FAKE, rank=FAKE, ids=FAKE, vals=FAKE)
    call = lambda **o: lib.ft_logprobs(*dict(ok, **o).values(), None, None)  # noqa: E731
    assert call(N=0) == ft.FT_OK
    assert call(top=33) == ft.FT_ERR_UNSUPPORTED and call(V=3, top=4) == ft.FT_ERR_UNSUPPORTED
    assert call(V=2 ** 30 + 1, stride=2 ** 31) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(x=None), dict(dt=2), dict(stride=99), dict(N=-1), dict(V=0), dict(top=-1), dict(ids=None), dict(vals=None),
                dict(t=None), dict(x=FAKE + 2), dict(x=FAKE + 1, dt=ft.FT_BF16)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad
