"""History cache without a GPU: what the entry points refuse before anything is
launched, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest

from oracle import cache_oracle as CO


@pytest.fixture(scope="module")
def svg():
    from video_dit_spatial_b200 import _build
    _build.build()
    import video_dit_spatial_b200 as m
    m.load()
    return m


def _geom(svg, n_pages=8, page_size=16, H_kv=2, d=64, max_seqs=4, max_pages=5):
    return svg.CacheGeom(n_pages, page_size, H_kv, d, max_seqs, max_pages)


# (entry point, arguments after the geometry that are fine as far as the host can tell)
CALLS = {
    "svg_cache_reset": [256, 256, 256, None],
    "svg_cache_fork": [256, 256, 256, 256, 256, 3, None],
    "svg_cache_free": [256, 256, 256, 256, None, 3, None],
    "svg_cache_reserve": [256, 256, 256, 256, 256, 3, 256, None],
    "svg_cache_write": [256, 256, 256, 3, 7, 256, 256, 256, 256, None],
    "svg_cache_compact": [256, 256, 256, 256, 256, None],
    "svg_cache_copy_pages": [256, 4, 256, 256, 256, 256, None],
    "svg_prefix_attention": [2, 4, 3, 0, 17, ctypes.c_float(0.1), 1 << 20, 256, 256, 256, 256, 256,
                             256, None, 256, 1 << 40, None],
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_bad_sizes_are_refused_before_the_device(svg, name):
    f = getattr(svg.load(), name)

    def status(**kw):
        return f(ctypes.byref(_geom(svg, **kw)), *CALLS[name])

    assert f(None, *CALLS[name]) == svg.SVG_ERR_INVALID_ARG
    for kw in (dict(n_pages=0), dict(H_kv=0), dict(max_seqs=0), dict(max_pages=-1),
               dict(n_pages=(1 << 24) + 1), dict(H_kv=65536),
               dict(max_pages=(1 << 26) + 1), dict(max_seqs=1 << 20, max_pages=1 << 12),
               dict(n_pages=1 << 24, H_kv=64)):
        assert status(**kw) == svg.SVG_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(page_size=8), dict(page_size=48), dict(page_size=512)):
        assert status(**kw) == svg.SVG_ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("name", sorted(CALLS))
def test_null_and_misaligned_pointers_are_refused(svg, name):
    f = getattr(svg.load(), name)
    g = _geom(svg)
    optional = {"svg_cache_free": {4}, "svg_prefix_attention": {13}}
    for at, x in enumerate(CALLS[name][:-1]):
        if not isinstance(x, int) or x < 256 or x == 1 << 40:
            if x is not None or at not in optional.get(name, set()):
                continue
        args = list(CALLS[name])
        args[at] = (x or 256) + 2  # every pointer is to at least 4-byte values
        assert f(ctypes.byref(g), *args) == svg.SVG_ERR_INVALID_ARG, (name, at)
        if x is not None:
            args[at] = None
            assert f(ctypes.byref(g), *args) == svg.SVG_ERR_INVALID_ARG, (name, at)


def test_list_lengths_and_shapes_are_refused(svg):
    lib = svg.load()
    g = _geom(svg)

    def call(name, **at):
        args = list(CALLS[name])
        for k, x in at.items():
            args[int(k[1:])] = x
        return getattr(lib, name)(ctypes.byref(g), *args)

    for n in (0, -1, 1025):
        assert call("svg_cache_fork", _5=n) == svg.SVG_ERR_INVALID_ARG
        assert call("svg_cache_free", _5=n) == svg.SVG_ERR_INVALID_ARG
        assert call("svg_cache_reserve", _5=n) == svg.SVG_ERR_INVALID_ARG
        assert call("svg_cache_write", _3=n) == svg.SVG_ERR_INVALID_ARG
    assert call("svg_cache_write", _4=0) == svg.SVG_ERR_INVALID_ARG
    for n in (0, 9):
        assert call("svg_cache_copy_pages", _1=n) == svg.SVG_ERR_INVALID_ARG
    for at in (dict(_0=0), dict(_0=1025), dict(_1=3), dict(_1=0), dict(_2=0), dict(_2=1 << 30),
               dict(_3=-1), dict(_3=4), dict(_4=-1), dict(_4=81),
               dict(_5=ctypes.c_float(0.0)), dict(_5=ctypes.c_float(float("nan"))),
               dict(_5=ctypes.c_float(float("inf"))),
               dict(_6=512),  # q overlaps o at 256
               dict(_14=256 + 16)):  # workspace alignment
        assert call("svg_prefix_attention", **at) == svg.SVG_ERR_INVALID_ARG, at
    need = svg.svg_prefix_attention_workspace_bytes(g, 2, 4, 3)
    assert need > 0
    assert call("svg_prefix_attention", _15=need - 1) == svg.SVG_ERR_CAPACITY
    with pytest.raises(svg.SvgError):
        svg.svg_prefix_attention_workspace_bytes(g, 2, 3, 3)


@pytest.mark.parametrize("H,H_kv,d", [(8, 8, 64), (8, 2, 128), (64, 1, 128), (40, 1, 64)])
def test_a_workspace_for_the_largest_call_serves_the_smaller_ones(svg, H, H_kv, d):
    g = _geom(svg, n_pages=1000, H_kv=H_kv, d=d)
    rows = [1, 2, 3, 4, 7, 16, 17, 31, 40, 64, 129, 200, 256, 257, 400, 513, 900, 2304, 2305, 5000]
    most = {}
    for B in (1, 2, 3, 5, 8, 17, 40, 300, 1024):
        before = 0
        for L in rows:
            n = svg.svg_prefix_attention_workspace_bytes(g, B, H, L)
            assert n >= before and n >= most.get(L, 0)
            most[L] = before = n


def test_binding_refuses_host_tensors(svg):
    import torch
    g = _geom(svg)
    table = torch.zeros(20, dtype=torch.int32)
    with pytest.raises(ValueError, match="device buffers"):
        svg.svg_cache_reset(g, table, table, table)


def test_attention_refuses_tables_of_longer_rows(svg):
    """Above 2^20 rows the bookkeeping goes on, the attention does not."""
    for ps in (16, 256):
        fits, over = (1 << 20) // ps, (1 << 20) // ps + 1
        assert svg.svg_prefix_attention_workspace_bytes(_geom(svg, page_size=ps, max_pages=fits),
                                                        2, 4, 3) > 0
        with pytest.raises(svg.SvgError) as e:
            svg.svg_prefix_attention_workspace_bytes(_geom(svg, page_size=ps, max_pages=over), 2, 4, 3)
        assert e.value.status == svg.SVG_ERR_INVALID_ARG


# ---------------------------------------------------------------- the oracle
def test_model_by_hand():
    m = CO.CacheModel(n_pages=6, page_size=16, H_kv=1, d=2, max_seqs=3, max_pages=3)
    assert m.reserve([0], [20]) == [[0, 20, -1, -1]]
    assert m.table[0].tolist() == [0, 1, -1] and m.refs.tolist() == [1, 1, 0, 0, 0, 0]
    m.fork([0, 0], [1, 2])
    assert m.refs.tolist() == [3, 3, 0, 0, 0, 0] and m.lens.tolist() == [20, 20, 20]
    # the open page is shared: both get their own; sequence 2 also grows by a page
    assert m.reserve([1, 2], [1, 13]) == [[20, 1, 1, 2], [20, 13, 1, 3]]
    assert m.table.tolist() == [[0, 1, -1], [0, 2, -1], [0, 3, 4]]
    assert m.refs.tolist() == [3, 1, 1, 1, 1, 0]
    m.free([0])
    assert m.refs.tolist() == [2, 0, 1, 1, 1, 0]
    assert m.compact() == [(4, 1)]
    assert m.table.tolist() == [[-1, -1, -1], [0, 2, -1], [0, 3, 1]]
    m.check()
    # two free pages left: three are not handed out, and nothing else is
    before = m.table.copy()
    assert m.reserve([0, 1], [17, 12]) == [[0, 0, -1, -1], [21, 0, -1, -1]]
    assert m.bits == 4 and np.array_equal(m.table, before)


def test_forks_and_frees_give_every_page_back():
    rng = np.random.default_rng(1)
    m = CO.CacheModel(40, 16, 1, 2, 6, 8)
    for _ in range(200):
        s = int(rng.integers(6))
        what = rng.integers(4)
        if what == 0 and m.lens[s] == 0:
            src = [x for x in range(6) if x != s]
            m.fork([src[int(rng.integers(5))]], [s])
        elif what == 1:
            m.free([s], [int(rng.integers(0, 40))])
        elif what == 2:
            m.reserve([s], [int(rng.integers(0, 30))])
        else:
            m.compact()
        m.check()
    m.free(list(range(6)))
    assert not m.refs.any() and not m.lens.any()


def test_prefix_attention_is_attention_over_the_joined_rows():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 9, 2, 16, 4))
    q = rng.standard_normal((2, 4, 3, 4))
    table = np.array([[4, 2, -1], [4, 7, 1], [4, 0, -1]])
    lens = [20, 40, 20]
    o, lse, _ = CO.prefix_attention(q, k, v, table, lens, [1, 2], 0, 20, 0.5, 16)
    for b, (s, own) in enumerate([(1, range(20, 40)), (2, [])]):
        where = [(0, p) for p in range(20)] + [(s, p) for p in own]
        for h in range(4):
            kk, vv = (np.array([x[table[t, p // 16], h // 2, p % 16] for t, p in where])
                      for x in (k, v))
            w = np.exp(0.5 * q[b, h] @ kk.T)
            np.testing.assert_allclose(o[b, h], (w / w.sum(1, keepdims=True)) @ vv, rtol=1e-12)
            np.testing.assert_allclose(lse[b, h], np.log(w.sum(1)), rtol=1e-12)
