"""GPU parity of the history cache against its oracle: page tables, lengths,
counts, plans, moves and the rows themselves are whole values or copies, so
everything is compared for equality."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svg():
    import video_dit_spatial_b200 as m
    m.load()
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """The library's cache and the oracle's, driven by the same calls."""

    def __init__(self, svg, n_pages, ps, H_kv, d, max_seqs, max_pages, seed=0):
        self.svg = svg
        self.geom = svg.CacheGeom(n_pages, ps, H_kv, d, max_seqs, max_pages)
        self.m = CO.CacheModel(n_pages, ps, H_kv, d, max_seqs, max_pages)
        rng = np.random.default_rng(seed)
        self.m.k[:] = rng.integers(-2 ** 15, 2 ** 15, self.m.k.shape)  # every bit pattern, NaN too
        self.m.v[:] = rng.integers(-2 ** 15, 2 ** 15, self.m.v.shape)
        self.rng = rng
        self.k, self.v = (torch.from_numpy(x.copy()).cuda().view(torch.bfloat16)
                          for x in (self.m.k, self.m.v))
        self.table = torch.full((max_seqs, max_pages), 99, dtype=torch.int32, device="cuda")
        self.lens, self.refs = dev([7] * max_seqs), dev([3] * n_pages)
        self.moves = torch.zeros(2 + 2 * n_pages, dtype=torch.int32, device="cuda")
        svg.svg_cache_reset(self.geom, *self.state)

    @property
    def state(self):
        return self.table, self.lens, self.refs

    def fork(self, src, dst):
        self.svg.svg_cache_fork(self.geom, *self.state, dev(src), dev(dst))
        self.m.fork(src, dst)

    def free(self, seqs, keep=None):
        self.svg.svg_cache_free(self.geom, *self.state, dev(seqs), None if keep is None else dev(keep))
        self.m.free(seqs, keep)

    def append(self, seqs, counts, L=None):
        plan = torch.full((len(seqs), 4), -9, dtype=torch.int32, device="cuda")
        self.svg.svg_cache_reserve(self.geom, *self.state, dev(seqs), dev(counts), plan)
        want = self.m.reserve(seqs, counts)
        got = plan.tolist()
        for s, g, w in zip(seqs, got, want):
            if w[1] or w[2] >= 0:
                assert g == w
            else:
                assert g[1:] == w[1:]
        L = max([1] + list(counts)) if L is None else L
        shape = (len(seqs), self.geom.H_kv, L, self.geom.head_dim)
        rows = [self.rng.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16) for _ in range(2)]
        new = [torch.from_numpy(x).cuda().view(torch.bfloat16) for x in rows]
        self.svg.svg_cache_write(self.geom, self.table, dev(seqs), plan, L, *new, self.k, self.v)
        self.m.write(seqs, want, *rows)

    def compact(self, in_place=True):
        out = (self.table, self.refs) if in_place else (torch.full_like(self.table, 77),
                                                        torch.full_like(self.refs, 77))
        self.svg.svg_cache_compact(self.geom, self.table, self.refs, *out, self.moves)
        self.svg.svg_cache_copy_pages(self.geom, self.moves, self.geom.n_pages, self.k, self.v,
                                      self.k, self.v)
        self.table, self.refs = out
        want = self.m.compact()
        got = self.moves.tolist()
        assert got[0] == len(want) and got[1] == int((self.m.refs > 0).sum())
        assert [tuple(got[2 + 2 * i:4 + 2 * i]) for i in range(got[0])] == want

    def check(self, bits=0):
        _, got = self.svg.svg_get_device_status()
        assert got == self.m.bits == bits
        self.m.bits = 0
        assert np.array_equal(self.table.cpu().numpy(), self.m.table)
        assert np.array_equal(self.lens.cpu().numpy(), self.m.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.m.refs)
        assert np.array_equal(self.k.view(torch.int16).cpu().numpy(), self.m.k)
        assert np.array_equal(self.v.view(torch.int16).cpu().numpy(), self.m.v)
        self.m.check()


def test_reset(svg):
    b = Both(svg, 37, 16, 1, 64, 5, 3)
    b.check()


@pytest.mark.parametrize("ps,H_kv,d", [(16, 3, 64), (32, 1, 128), (64, 2, 64), (128, 5, 128),
                                       (256, 2, 128)])
def test_a_run_of_steps(svg, ps, H_kv, d):
    b = Both(svg, 60, ps, H_kv, d, 7, 6, seed=ps)
    b.append([0], [2 * ps + 5])
    b.check()
    b.fork([0, 0, -1, 0], [1, 2, 3, 4])
    b.append([1, -1, 2, 4], [1, 4, ps, 0])  # copies of the open page; one entry adds nothing
    b.check()
    b.append([1, 2, 0], [ps - 6, 1, ps - 5])  # to the end of a page, past one, in place
    b.check()
    b.fork([2], [5])
    b.free([2, 1], [ps + 1, ps])  # cut inside a shared page, and at the end of one
    b.append([2, 5], [3, 2])
    b.check()
    b.free([0, -1, 4])
    b.compact(in_place=False)
    b.check()
    b.append([0, 1, 2, 3, 5], [ps, 2 * ps, 1, 1, 7], L=2 * ps + 3)
    b.free([5])
    b.compact()
    b.compact()  # nothing left to move
    b.check()


@pytest.mark.parametrize("seed", range(3))
def test_random_steps(svg, seed):
    rng = np.random.default_rng(100 + seed)
    b = Both(svg, 90, 16, 2, 64, 12, 9, seed=seed)
    for _ in range(60):
        seqs = rng.permutation(12)[:int(rng.integers(1, 7))].tolist()
        what = int(rng.integers(4))
        if what == 0:
            empty = [s for s in range(12) if b.m.lens[s] == 0]
            rest = [s for s in range(12) if s not in empty]
            if empty and rest:
                b.fork([int(rng.choice(rest)) for _ in empty[:3]], empty[:3])
        elif what == 1:
            b.free(seqs, [int(x) for x in rng.integers(0, 140, len(seqs))])
        elif what == 2:
            b.append(seqs, [int(x) for x in rng.integers(0, 50, len(seqs))])
        else:
            b.compact(in_place=bool(rng.integers(2)))
        b.check(b.m.bits)  # the pool runs out at times


def test_many_entries_and_a_long_pool(svg):
    """More pages than one pass over the counts sees, and a full list."""
    b = Both(svg, 40000, 16, 1, 64, 1100, 40, seed=3)
    rng = np.random.default_rng(4)
    b.append(list(range(1024)), [int(x) for x in rng.integers(300, 640, 1024)])
    b.free([int(s) for s in rng.permutation(1100)[:700]])
    b.check()
    b.append(list(range(500, 1100)), [int(x) for x in rng.integers(0, 40, 600)])
    b.check(b.m.bits)
    b.compact()
    b.check()


def test_no_room_leaves_everything(svg):
    b = Both(svg, 6, 16, 1, 64, 4, 5)
    b.append([0], [70])  # five pages
    b.check()
    b.append([1, 2], [16, 1])  # two wanted, one free
    b.check(bits=4)
    b.append([1, 0], [16, 11])  # past the table's width: the other entry is served
    b.check(bits=4)
    b.append([1, 2, 3], [0, 0, 0])
    b.check()


def test_more_pages_wanted_than_an_int_counts(svg):
    """1024 entries that want 2^22 + 1 pages each, 2^32 + 1024 between them: nothing is reserved."""
    width = (1 << 22) + 1
    geom = svg.CacheGeom(64, 256, 1, 64, 1025, 1 << 20)
    small = svg.CacheGeom(64, 16, 1, 64, 505, width)  # 505 * width entries fit 2^31
    for g, counts in ((geom, (1 << 20) * 256), (small, 16 * width)):
        n = min(1024, g.max_seqs)
        table = torch.full((g.max_seqs, g.max_pages), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(g.max_seqs, dtype=torch.int32, device="cuda")
        refs = torch.zeros(64, dtype=torch.int32, device="cuda")
        plan = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
        seqs = torch.arange(n, dtype=torch.int32, device="cuda")
        svg.svg_cache_reserve(g, table, lens, refs, seqs, torch.full_like(seqs, counts), plan)
        assert svg.svg_get_device_status()[1] == 4
        assert not lens.any() and not refs.any() and torch.all(table == -1)
        assert torch.all(plan[:, 1] == 0) and torch.all(plan[:, 2:] == -1)
        del table


def test_refused_entries_change_nothing(svg):
    b = Both(svg, 20, 16, 1, 64, 5, 3)
    b.append([0, 1], [20, 5])
    b.fork([0, 0, 1], [2, 2, 1])  # the same target twice; a target that is a source and not empty
    b.check(bits=2)
    b.fork([0, 9, 0], [3, 4, 7])  # numbers past the table
    b.check(bits=2)
    b.fork([4, 0], [1, 0])  # an empty source is fine, a target in use is not
    b.check(bits=2)
    b.free([0, 0, 8, 1], [1, 0, 0, -3])
    b.check(bits=2)
    b.append([1, 1, 6, 0], [3, 9, 2, -1])
    b.check(bits=2)


def test_a_state_that_cannot_be_is_flagged_not_followed(svg):
    b = Both(svg, 8, 16, 1, 64, 3, 4)
    b.append([0, 1], [20, 20])
    b.check()
    keep = [x.clone() for x in (b.k, b.v)]
    bad = dev([8, 1 << 30])
    b.table[0, :2] = bad
    plan = torch.tensor([[20, 3, -1, -1]], dtype=torch.int32, device="cuda")
    new = torch.ones((1, 1, 3, 64), dtype=torch.bfloat16, device="cuda")
    seq = dev([0])
    for call in (lambda: svg.svg_cache_write(b.geom, b.table, seq, plan, 3, new, new, b.k, b.v),
                 lambda: svg.svg_cache_reserve(b.geom, *b.state, seq, dev([1]), plan),
                 lambda: svg.svg_cache_fork(b.geom, *b.state, seq, dev([2])),
                 lambda: svg.svg_cache_free(b.geom, *b.state, seq)):
        call()
        assert svg.svg_get_device_status()[1] == 2
    # a plan that does not fit the rows, and moves past the pool or past the list
    for p in ([[0, 4, -1, -1]], [[-1, 2, -1, -1]], [[63, 2, -1, -1]], [[0, 1, 8, 1]], [[0, 1, -1, 1]]):
        svg.svg_cache_write(b.geom, b.table, dev([1]), dev(p), 3, new, new, b.k, b.v)
        assert svg.svg_get_device_status()[1] == 2
    for moves in ([2, 0, 8, 1, -1, 3], [-4, 0, 1, 2, 1, 2]):
        svg.svg_cache_copy_pages(b.geom, dev(moves), 2, b.k, b.v, b.k, b.v)
        assert svg.svg_get_device_status()[1] == 2
    written = int(b.m.table[1, 0])
    rest = [p for p in range(8) if p != written]
    assert all(torch.equal(x.view(torch.int16)[rest], y.view(torch.int16)[rest])
               for x, y in zip(keep, (b.k, b.v)))


def test_copy_between_pools(svg):
    b = Both(svg, 9, 32, 3, 128, 1, 1)
    k2, v2 = torch.zeros_like(b.k), torch.zeros_like(b.v)
    svg.svg_cache_copy_pages(b.geom, dev([3, 0, 8, 0, 2, 4, 5, 5]), 3, b.k, b.v, k2, v2)
    for x, y in ((b.k, k2), (b.v, v2)):
        x, y = x.view(torch.int16), y.view(torch.int16)
        assert all(torch.equal(x[i], y[j]) for i, j in ((8, 0), (2, 4), (5, 5)))
        assert not y[[1, 2, 3, 6, 7, 8]].any()
    assert svg.svg_get_device_status()[1] == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_drops_table_entries_that_name_no_page_in_use(svg, in_place):
    """Free pages below and above the number of pages in use, and pages past the pool."""
    geom = svg.CacheGeom(40, 16, 1, 64, 3, 8)
    refs = [0] * 40
    for p in (0, 2, 3, 20, 39):
        refs[p] = 1
    #        in use           free       past the pool; none
    table = [[0, 20, 3, 39] + [1, 4] + [40, -1],
             [2, 39, 0, 2] + [21, 38] + [2 ** 30, -1],
             [-1] * 8]
    t, r = dev(table), dev(refs)
    out = (t, r) if in_place else (torch.full_like(t, 77), torch.full_like(r, 77))
    moves = torch.zeros(2 + 2 * 40, dtype=torch.int32, device="cuda")
    svg.svg_cache_compact(geom, t, r, *out, moves)
    st, bits = svg.svg_get_device_status()
    assert st == svg.SVG_ERR_INVALID_ARG and bits == 2
    assert moves[:6].tolist() == [2, 5, 20, 1, 39, 4]
    assert out[0].tolist() == [[0, 1, 3, 4] + [-1] * 4, [2, 4, 0, 2] + [-1] * 4, [-1] * 8]
    assert out[1].tolist() == [1] * 5 + [0] * 35


def test_history_cache_refuses_a_plan_of_an_earlier_state(svg):
    from video_dit_spatial_b200.layer import HistoryCache
    cache = HistoryCache(1, 8, 16, 1, 1, 64, 4, 64, 2, 8)
    k = torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    for change in (lambda: cache.fork(dev([0]), dev([1])), lambda: cache.free(dev([1])),
                   cache.compact, cache.reset):
        cache.reserve(dev([0]), dev([8]))
        cache.write(0, k, k)
        cache.write(0, k, k)
        change()
        with pytest.raises(ValueError, match="follows reserve"):
            cache.write(0, k, k)
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)


def test_history_cache_refuses_other_shapes(svg):
    from video_dit_spatial_b200.layer import HistoryCache
    cache = HistoryCache(1, 8, 16, 4, 2, 64, 4, 64, 2, 8)
    seqs = dev([0, 1])
    new = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cache.reserve(seqs, dev([8, 8]))
    cache.write(0, new(2, 2, 8, 64), new(2, 2, 8, 64))
    for k, v in ((new(2, 4, 8, 64), new(2, 4, 8, 64)), (new(2, 2, 8, 128), new(2, 2, 8, 128)),
                 (new(3, 2, 8, 64), new(3, 2, 8, 64)), (new(2, 2, 8, 64), new(2, 2, 9, 64))):
        with pytest.raises(ValueError, match="rows of shape"):
            cache.write(0, k, v)
    q, o, lse = new(2, 4, 8, 64), new(2, 4, 8, 64), torch.zeros((2, 4, 8), device="cuda")
    cache.attend(0, q, seqs, 0, 0, o, lse)
    assert torch.all(o == 0) and torch.all((lse - np.log(8.0)).abs() < 1e-5)
    for bad in ((new(2, 8, 8, 64), new(2, 8, 8, 64), None), (q, new(2, 4, 9, 64), None),
                (new(3, 4, 8, 64), new(3, 4, 8, 64), None), (q, o, lse[:, :, :4])):
        with pytest.raises(ValueError, match="queries of shape"):
            cache.attend(0, bad[0], seqs, 0, 0, *bad[1:])
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)
