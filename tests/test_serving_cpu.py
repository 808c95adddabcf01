"""Rows of the fused projection, draft trees, moved entries and prompt attention without a GPU: the
oracle's pins and the refusals of the entry points (every call here returns before a launch)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

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
def test_tree_rows_hand_case():
    #   0 - 1 - 3
    #     \ 2        4 is another root
    see = paged.tree_rows([-1, 0, 0, 1, -1])
    want = [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    np.testing.assert_array_equal(see, np.array(want, bool))
    assert paged.mask_words(see, 1)[:, 0].tolist() == [1, 3, 5, 11, 16]
    wide = np.zeros((1, 40), bool)
    wide[0, [0, 31, 32, 39]] = True
    assert paged.mask_words(wide, 2).tolist() == [[-(1 << 31) + 1, 1 + 128]]


def test_attend_seen_is_attend_rows():
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=(4, 64)), g.normal(size=(9, 64)), g.normal(size=(9, 64))
    seen = np.arange(9)[None, :] <= 5 + np.arange(4)[:, None]
    for a, b in zip(paged.attend_seen(q, k, v, 32, 0.1, seen), paged.attend_rows(q, k, v, 32, 0.1, 5)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-14)
    seen[2] = False
    assert not paged.attend_seen(q, k, v, 32, 0.1, seen)[0][2].any()


def test_norm_rope_closed_forms():
    x = np.full((1, 64), 3.0)
    np.testing.assert_allclose(paged.norm_rope(x, np.full(64, 2.0), 0, 1e4, 0.0), np.full((1, 64), 2.0))
    g = np.random.default_rng(1)
    y = g.normal(size=(2, 128))
    z = paged.norm_rope(y, None, 7, 1e4, 1e-5)
    np.testing.assert_allclose(np.linalg.norm(z, axis=-1), np.linalg.norm(y, axis=-1))
    c = (y[:, :64] + 1j * y[:, 64:]) * np.exp(7j * 1e4 ** (-np.arange(64) / 64))
    np.testing.assert_allclose(z, np.concatenate([c.real, c.imag], -1), atol=1e-12)


# ---------------------------------------------------------------- refusals
def _caller(name, ft, c, ok, tail):
    fn = getattr(ft.lib(), name)
    return lambda **o: fn(ctypes.byref(c), *dict(ok, **o).values(), *tail)


def test_norm_rope_refusals(ft):
    c = ft.cfg_from_shape(synth.L8B)
    ok = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, gq=None, gk=None, pos=FAKE, total=3, qo=FAKE, qos=4096, ko=FAKE, kos=1024)
    call = _caller("ft_qk_norm_rope_bf16", ft, c, ok, (None,))
    assert call(total=0) == ft.FT_OK and call(total=0, q=None, qo=None) == ft.FT_OK
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=None, qo=None, k=None, ko=None), dict(total=-1),
                dict(pos=None), dict(qs=4095), dict(ks=1023), dict(qos=4095), dict(kos=0)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad
    call = _caller("ft_qk_norm_rope_bf16", ft, ft.make_cfg(512, 8, 2, 96, 512, had_block=32), ok, (None,))
    assert call() == ft.FT_ERR_UNSUPPORTED


def test_append_rope_refusals(ft):
    c = ft.cfg_from_shape(synth.L8B)
    ok = dict(pages=FAKE, n=8, ps=64, k=FAKE, ks=1024, v=FAKE, vs=1024, gk=None, pos=FAKE, slots=FAKE, total=3, q=None, qs=0,
              gq=None, qo=None, qos=0)
    call = _caller("ft_kv_append_rope_paged_int4", ft, c, ok, (None, None))
    assert call(total=0) == ft.FT_OK and call(ps=8) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(pages=None), dict(pages=FAKE + 8), dict(n=0), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None),
                dict(total=-1), dict(ks=1023), dict(vs=0), dict(q=FAKE), dict(qo=FAKE), dict(q=FAKE, qo=FAKE, qs=4096, qos=4095),
                dict(q=FAKE, qo=FAKE, qs=100, qos=4096)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_move_refusals(ft):
    c = ft.cfg_from_shape(synth.L8B)
    ok = dict(pages=FAKE, n=8, ps=64, src=FAKE, dst=FAKE, B=2, m=4)
    call = _caller("ft_kv_move_paged_int4", ft, c, ok, (None, None))
    assert call(B=0) == ft.FT_OK and call(m=0) == ft.FT_OK
    assert call(ps=48) == ft.FT_ERR_UNSUPPORTED and call(m=257) == ft.FT_ERR_UNSUPPORTED and call(B=2 ** 29) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(pages=None), dict(pages=FAKE + 4), dict(n=0), dict(src=None), dict(dst=None), dict(B=-1), dict(m=-1)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_tree_refusals(ft):
    c = ft.cfg_from_shape(synth.L8B)
    size = ft.ft_attn_tree_workspace_bytes(c, 4, 100, 40)
    assert size > 0 and ft.ft_attn_tree_workspace_bytes(c, 0, 100, 40) == 0 and ft.ft_attn_tree_workspace_bytes(c, 4, 100, 0) == 0
    ok = dict(pages=FAKE, n=8, ps=64, q=FAKE, qs=4096, cu=FAKE, kv=FAKE, table=FAKE, stride=4, mask=FAKE, ms=2, B=4, total=100,
              max_q=40, scale=0.1, o=FAKE, os=4096, ws=FAKE, wsb=size)
    call = _caller("ft_attn_tree_paged_int4", ft, c, ok, (None, None))
    assert call(total=0) == ft.FT_OK and call(wsb=size - 1) == ft.FT_ERR_WORKSPACE and call(ps=40) == ft.FT_ERR_UNSUPPORTED
    for big in (dict(total=2 ** 29), dict(stride=2 ** 28), dict(B=8193)):
        assert call(wsb=2 ** 60, **big) == ft.FT_ERR_UNSUPPORTED, big
    # what grows with the rows: blocks of 256, rows of the batch, rows of the call
    for big in (dict(B=4096, stride=2048, max_q=2000, total=2000, ms=63), dict(B=8192, stride=1, max_q=2 ** 15, total=2 ** 15, ms=1024),
                dict(B=1, stride=1, total=2 ** 26, max_q=100, ms=4)):
        assert call(wsb=2 ** 60, **big) == ft.FT_ERR_UNSUPPORTED, big
    for bad in (dict(pages=None), dict(q=None), dict(o=None), dict(cu=None), dict(kv=None), dict(table=None), dict(ws=None),
                dict(ws=FAKE + 4), dict(B=0), dict(total=-1), dict(max_q=0), dict(stride=0), dict(qs=4095), dict(os=1),
                dict(scale=0.0), dict(scale=float("nan")), dict(mask=None), dict(mask=FAKE + 2), dict(ms=1), dict(ms=0)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad


def test_tree_workspace_grows(ft):
    """A workspace for the longest trees is enough for shorter ones, whichever kernel takes them."""
    for n_q, n_kv, d in ((32, 8, 128), (8, 8, 64), (56, 7, 128)):
        c = ft.make_cfg(n_q * d, n_q, n_kv, d, 1024)
        for B, total in ((1, 600), (40, 900)):
            sizes = [ft.ft_attn_tree_workspace_bytes(c, B, total, q) for q in range(1, 600)]
            assert sizes == sorted(sizes) and sizes[-1] <= ft.ft_attn_tree_workspace_bytes(c, B + 1, total + 1, 600)


def test_prompt_refusals(ft):
    c = ft.cfg_from_shape(synth.L8B)
    ok = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, cu=FAKE, B=4, total=100, max_len=40, scale=0.1, o=FAKE, os=4096)
    call = _caller("ft_attn_prompt_bf16", ft, c, ok, (None, None))
    assert call(total=0) == ft.FT_OK
    assert call(B=8193) == ft.FT_ERR_UNSUPPORTED and call(total=2 ** 29) == ft.FT_ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(cu=None), dict(B=0), dict(total=-1), dict(max_len=0),
                dict(qs=4095), dict(ks=1023), dict(vs=1023), dict(os=0), dict(scale=0.0), dict(scale=float("inf")), dict(k=FAKE + 8),
                dict(v=FAKE + 2), dict(ks=1028), dict(vs=1025), dict(q=FAKE + 2), dict(qs=4100)):
        assert call(**bad) == ft.FT_ERR_INVALID_ARG, bad
    assert call(ks=2 ** 40) == ft.FT_ERR_UNSUPPORTED


# ---------------------------------------------------------------- what an item of prompt attention is
WALK = r"""
#include "ft_prompt_items.h"
// blocks[n] of each sequence, items[k] in any order -> (sequence, place) of each; -1: none
extern "C" void walk(const int* blocks, int n, const int* items, int k, int* out) {
  int top = -1;
  for (int b = 0; b < n; ++b) top = blocks[b] - 1 > top ? blocks[b] - 1 : top;
  ft::ItemWalk w(top);
  auto have = [&](int level) {
    uint32_t bits = 0;
    for (int b = 0; b < n; ++b) bits |= (uint32_t)(blocks[b] > level) << b;
    return bits;
  };
  for (int i = 0; i < k; ++i) {
    const uint32_t some = w.find(items[i], have, [](uint32_t bits) { return __builtin_popcount(bits); });
    int at = items[i] - w.above, b = at < 0 ? n : 0;
    for (; b < n; ++b)
      if ((some >> b & 1) && at-- == 0) break;
    out[2 * i] = b < n ? b : -1, out[2 * i + 1] = w.level;
  }
}
"""


@pytest.fixture(scope="module")
def item_walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("walk")
    (at / "walk.cpp").write_text(WALK)
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_weight_kv_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, "-o", str(at / "walk.so"), str(at / "walk.cpp")], check=True)
    fn = ctypes.CDLL(str(at / "walk.so")).walk

    def run(blocks, items):
        out = np.full((len(items), 2), -9, np.int32)
        ptr = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_int))  # noqa: E731
        b, i = (np.ascontiguousarray(x, np.int32) for x in (blocks, items))
        fn(ptr(b), len(b), ptr(i), len(i), ptr(out))
        return [tuple(x) for x in out.tolist()]
    return run


@pytest.mark.parametrize("blocks", [[1], [4], [3, 1, 0, 5, 5], [0, 0, 2], [1] * 32, list(range(32)), [40, 1, 39, 2]])
def test_prompt_items_in_any_order(item_walk, blocks):
    """An item is the same block whatever items came before it: ascending, descending, shuffled, the same one again."""
    want = [(b, level) for level in range(max(blocks) - 1, -1, -1) for b, n in enumerate(blocks) if n > level]
    n, g = len(want), np.random.default_rng(len(blocks))
    up = np.arange(n)
    for items in (up, up[::-1], up[::2], g.permutation(n), g.integers(0, n, 200), np.repeat(up, 2)):
        assert item_walk(blocks, items) == [want[i] for i in items]
