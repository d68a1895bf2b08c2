"""What a history cache's calls leave behind where the state holds a page number that cannot be."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svg():
    import video_dit_spatial_b200 as m
    m.load()
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(svg, width, n_pages, bad_slot, bad_page):
    """Sequence 0 has `width` pages of 16 rows, one of which is not a page; 1 is a good one of
    two pages that it shares with 0; 2 and 3 are empty."""
    geom = svg.CacheGeom(n_pages, 16, 1, 64, 4, width)
    table = torch.full((4, width), -1, dtype=torch.int32)
    table[0] = torch.arange(width)
    table[1, :2] = table[0, :2]
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[:width] = 1
    refs[:2] = 2
    table[0, bad_slot] = bad_page
    return geom, [table.cuda(), dev([16 * width - 3, 32, 0, 0]), refs.cuda()]


@pytest.mark.parametrize("width,bad_slot,bad_page", [(5, 4, 8), (5, 2, -1), (3000, 2999, 1 << 30),
                                                     (3000, 0, -7)])
def test_fork_of_a_bad_source_changes_nothing(svg, width, bad_slot, bad_page):
    geom, st = state(svg, width, width + 3, bad_slot, bad_page)
    before = [x.clone() for x in st]
    svg.svg_cache_fork(geom, *st, dev([0]), dev([2]))
    assert svg.svg_get_device_status()[1] == 2
    assert all(torch.equal(x, y) for x, y in zip(st, before))
    # the other entries of the call are served
    svg.svg_cache_fork(geom, *st, dev([0, 1]), dev([2, 3]))
    assert svg.svg_get_device_status()[1] == 2
    before[0][3] = before[0][1]
    before[1][3] = 32
    before[2][:2] += torch.tensor([0 <= p < width + 3 for p in before[0][1, :2].tolist()],
                                  device="cuda")
    assert all(torch.equal(x, y) for x, y in zip(st, before))


@pytest.mark.parametrize("width,bad_slot,bad_page", [(5, 4, 8), (5, 2, -1), (3000, 2999, 1 << 30)])
def test_free_passes_over_a_bad_page(svg, width, bad_slot, bad_page):
    """So that a sequence with one can be dropped: its other pages are given up."""
    geom, st = state(svg, width, width + 3, bad_slot, bad_page)
    svg.svg_cache_free(geom, *st, dev([0]))
    assert svg.svg_get_device_status()[1] == 2
    assert torch.all(st[0][0] == -1) and st[1].tolist() == [0, 32, 0, 0]
    refs = torch.zeros(width + 3, dtype=torch.int32)
    refs[:2] = 1
    if 0 <= bad_slot < width:
        refs[bad_slot] += 1  # the page that the entry should have named
    assert torch.equal(st[2].cpu(), refs)


def test_free_leaves_a_count_of_zero(svg):
    geom, st = state(svg, 5, 8, 4, 7)  # page 7 is free
    svg.svg_cache_free(geom, *st, dev([0]))
    assert svg.svg_get_device_status()[1] == 2
    assert st[2].tolist() == [1, 1, 0, 0, 1, 0, 0, 0]


@pytest.mark.parametrize("plan", [[0, 1, 8, 1], [0, 1, 1, 8], [0, 1, -1, 1], [0, 1, 1, -5], [3, 9, -1, -1],
                                  [-1, 2, -1, -1], [78, 3, -1, -1], [0, -1, 0, 1]])
def test_write_of_a_bad_plan_writes_nothing(svg, plan):
    geom, st = state(svg, 5, 8, 4, 4)
    pools = [torch.randn((8, 1, 16, 64), device="cuda").to(torch.bfloat16) for _ in range(2)]
    before = [x.clone() for x in pools]
    new = torch.ones((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    svg.svg_cache_write(geom, st[0], dev([0, 1]), dev([plan, [5, 2, -1, -1]]), 8, new, new, *pools)
    assert svg.svg_get_device_status()[1] == 2
    for x, y in zip(pools, before):
        y[0, :, 5:7] = 1.0  # the other entry of the call
        assert torch.equal(x, y)


@pytest.mark.parametrize("n,width", [(4, 1 << 16), (1024, 257), (1, 40)])
def test_far_more_pages_wanted_than_there_are(svg, n, width):
    """Every entry wants its whole table row: nothing is reserved; what is free can be had after."""
    geom = svg.CacheGeom(37, 16, 1, 64, n, width)
    st = [torch.full((n, width), -1, dtype=torch.int32, device="cuda"), dev([0] * n), dev([0] * 37)]
    seqs, plan = torch.arange(n, dtype=torch.int32, device="cuda"), dev([[9] * 4] * n)
    svg.svg_cache_reserve(geom, *st, seqs, torch.full_like(seqs, 16 * width), plan)
    assert svg.svg_get_device_status()[1] == 4
    assert torch.all(st[0] == -1) and not st[1].any() and not st[2].any()
    assert torch.equal(plan.cpu(), torch.tensor([[0, 0, -1, -1]] * n, dtype=torch.int32))
    counts = torch.zeros_like(seqs)
    counts[n - 1] = 16 * 37
    svg.svg_cache_reserve(geom, *st, seqs, counts, plan)
    assert svg.svg_get_device_status()[1] == 0
    assert st[0][n - 1, :37].tolist() == list(range(37)) and torch.all(st[2] == 1)
    assert plan[n - 1].tolist() == [0, 16 * 37, -1, -1] and st[1].tolist() == counts.tolist()
