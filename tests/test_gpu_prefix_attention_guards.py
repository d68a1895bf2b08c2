"""Nothing is written beside what a call is given: workspace, outputs and pools lie in
larger buffers whose other bytes are known. And the division of many short items, which
is limited in how many each CTA takes whole."""
import pytest
import torch

from test_gpu_prefix_attention import CASES, DEALT, Case, dev

pytestmark = pytest.mark.gpu

GUARD = 1 << 20  # bytes before and after


@pytest.fixture(scope="module")
def svg():
    import video_dit_spatial_b200 as m
    m.load()
    return m


class Guarded:
    """A tensor inside a buffer of 0xA5."""

    def __init__(self, shape, dtype, like=None):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        self.all = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.all[GUARD:GUARD + n].view(dtype).view(shape)
        if like is not None:
            self.t.copy_(like)

    def check(self):
        assert torch.all(self.all[:GUARD] == 0xA5) and torch.all(self.all[self.all.numel() - GUARD:] == 0xA5)


# few rows; beside gathered ones; gathered; the prefix in each sequence's items; dealt out
SHAPES = {name: CASES[name] for name in
          ("one_key", "one_row_long", "long_tails", "ends_inside_a_page", "grouped", "batch_300",
           "tiles_cross_sequences", "many_rows_each", "rows_129", "rows_257", "rows_700",
           "second_tile_of_few_rows")}
SHAPES.update(DEALT)


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_only_the_outputs_and_the_workspace_are_written(svg, name):
    c = Case(svg, *SHAPES[name], seed=31).call(svg)
    B, H, Lq, d = c.q.shape
    need = svg.svg_prefix_attention_workspace_bytes(c.geom, B, H, Lq)
    o, lse = Guarded(c.q.shape, torch.bfloat16), Guarded((B, H, Lq), torch.float32)
    ws = Guarded((need,), torch.uint8)
    inputs = [Guarded(x.shape, x.dtype, x) for x in (c.dq, c.dk, c.dv, *c.args[10:13])]
    before = [x.all.clone() for x in inputs]
    args = list(c.args)
    args[7:13], args[13], args[14] = [x.t for x in inputs], o.t, lse.t
    svg.svg_prefix_attention(*args, ws.t)
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)
    for x in (o, lse, ws):
        x.check()
    assert all(torch.equal(x.all, y) for x, y in zip(inputs, before))
    assert torch.equal(o.t, c.o) and torch.equal(lse.t, c.lse)


@pytest.mark.parametrize("name", ["one_row_long", "grouped", "tiles_cross_sequences", "many_rows_each"])
def test_a_smaller_call_in_the_workspace_of_a_larger_one(svg, name):
    """Just after a larger call left its pieces there: another form, other places of the pieces."""
    B, H, H_kv, d, ps, prefix, Lq, tails = CASES[name]
    c = Case(svg, *CASES[name], seed=32)
    c.call(svg).compare(name)
    large = Case(svg, B, H, H_kv, d, ps, prefix, 300, tails, seed=33)
    large.call(svg)
    need = svg.svg_prefix_attention_workspace_bytes(c.geom, B, H, 300)
    ws, o = Guarded((need,), torch.uint8), c.o.clone()
    svg.svg_prefix_attention(*large.args, ws.t)
    c.o.fill_(3.0)
    svg.svg_prefix_attention(*c.args, ws.t)
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)
    ws.check()
    assert torch.equal(c.o, o)


@pytest.mark.parametrize("d,ps,H_kv", [(64, 16, 2), (128, 64, 1)])
def test_only_the_pools_are_written(svg, d, ps, H_kv):
    """To the first and the last page of the pool, rows that end inside a page, replaced pages."""
    n_pages = 5
    geom = svg.CacheGeom(n_pages, ps, H_kv, d, 3, 4)
    shape = (n_pages, H_kv, ps, d)
    pools = [Guarded(shape, torch.bfloat16, torch.randn(shape, device="cuda")) for _ in range(2)]
    state = [Guarded(s, torch.int32) for s in ((3, 4), (3,), (n_pages,))]
    plan, moves = Guarded((2, 4), torch.int32), Guarded((2 + 2 * n_pages,), torch.int32)
    st = [x.t for x in state]
    svg.svg_cache_reset(geom, *st)
    new = torch.randn((2, H_kv, 2 * ps, d), device="cuda").to(torch.bfloat16)
    svg.svg_cache_reserve(geom, *st, dev([0, -1]), dev([2 * ps - 3, 5]), plan.t)
    svg.svg_cache_write(geom, st[0], dev([0, -1]), plan.t, 2 * ps, new, new, *[x.t for x in pools])
    svg.svg_cache_fork(geom, *st, dev([0]), dev([2]))
    svg.svg_cache_reserve(geom, *st, dev([2, 0]), dev([ps + 3, 1]), plan.t)
    svg.svg_cache_write(geom, st[0], dev([2, 0]), plan.t, 2 * ps, new, new, *[x.t for x in pools])
    assert sorted(st[0][0, :2].tolist() + st[0][2, 1:3].tolist()) == [0, 2, 3, 4]
    svg.svg_cache_free(geom, *st, dev([0]))
    svg.svg_cache_compact(geom, *[st[0], st[2]], *[st[0], st[2]], moves.t)
    svg.svg_cache_copy_pages(geom, moves.t, n_pages, *[x.t for x in pools] * 2)
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)
    for x in (*pools, *state, plan, moves):
        x.check()
    assert st[0][2].tolist() == [0, 2, 1, -1]  # page 3 took the number of the replaced page 1
    k = pools[0].t
    at = [(int(st[0][2, p // ps]), p % ps) for p in range(3 * ps)]
    got = torch.stack([k[page, :, row] for page, row in at], 1)
    assert torch.equal(got[:, :2 * ps - 3], new[0, :, :2 * ps - 3])
    assert torch.equal(got[:, 2 * ps - 3:], new[0, :, :ps + 3])


# Many items of one block: more whole ones for a CTA than it may take in turn.
@pytest.mark.parametrize("args", [(60, 80, 80, 64, 16, 0, 20, [i % 101 for i in range(60)]),
                                  (61, 80, 80, 128, 64, 0, 17, [(i * 37) % 129 for i in range(61)])])
def test_more_whole_items_than_a_cta_takes(svg, args):
    Case(svg, *args, seed=34).call(svg).compare()
