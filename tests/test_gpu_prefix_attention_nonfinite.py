"""svg_prefix_attention on rows whose scores are not finite.

A NaN among a row's scores, or a score of +inf, makes the row's O and lse NaN, as the
formula does; a row whose every score is -inf has weights of zero and counts as a row
without keys (O = 0, lse = -inf). Neither depends on where the work was cut into pieces,
nor reaches another row: those keep their bits.
"""
import pytest
import torch

from test_gpu_prefix_attention import CASES, DEALT, Case

pytestmark = pytest.mark.gpu

# every form: few rows, few rows beside gathered ones, gathered, the prefix in each
# sequence's own items; those dealt out whole and those cut
FORMS = {name: CASES[name] for name in
         ("nothing_shared", "one_row_long", "ends_inside_a_page", "grouped", "many_rows_each",
          "tiles_cross_sequences", "rows_128", "rows_256", "rows_700")}
FORMS.update({name: DEALT[name] for name in ("own_and_prefix", "gathered")})


@pytest.fixture(scope="module")
def svg():
    import video_dit_spatial_b200 as m
    m.load()
    return m


def rows_with_keys(c):
    """[B, H, Lq] of truth values: the entry's sequence sees at least one key."""
    some = torch.tensor([s >= 0 and (c.prefix > 0 or c.lens[s] > c.prefix) for s in c.seqs])
    return some[:, None, None].expand(c.q.shape[:3]).cuda()


def same_elsewhere(c, o, lse, bad):
    assert torch.equal(c.o[~bad], o[~bad]) and torch.equal(c.lse[~bad], lse[~bad])


@pytest.mark.parametrize("name", sorted(FORMS))
def test_nan_query_rows(svg, name):
    c = Case(svg, *FORMS[name], seed=21).call(svg)
    o, lse = c.o.clone(), c.lse.clone()
    B, H, Lq, d = c.q.shape
    bad = torch.zeros((B, H, Lq), dtype=torch.bool)
    for b, h, i, channels in ((0, 0, 0, slice(None)), (B - 1, H - 1, Lq - 1, slice(d - 1, d)),
                              (B // 2, H // 2, Lq // 2, slice(3, 4))):
        c.q[b, h, i, channels] = float("nan")
        bad[b, h, i] = True
    bad = bad.cuda() & rows_with_keys(c)
    c.call(svg)
    assert torch.all(torch.isnan(c.o[bad]))
    assert torch.all(torch.isnan(c.lse[bad]))
    same_elsewhere(c, o, lse, bad)
    without = ~rows_with_keys(c)
    assert torch.all(c.o[without] == 0) and torch.all(c.lse[without] == -float("inf"))


@pytest.mark.parametrize("name", sorted(FORMS))
def test_one_nan_key(svg, name):
    """The last key of a sequence's own: all of its rows, and no other's."""
    c = Case(svg, *FORMS[name], seed=22).call(svg)
    o, lse = c.o.clone(), c.lse.clone()
    b = max(range(c.B), key=lambda b: c.lens[b + 1])
    last = c.lens[b + 1] - 1
    assert last >= c.prefix
    c.k[c.table[b + 1, last // c.ps], :, last % c.ps, 5] = float("nan")
    c.call(svg)
    bad = torch.zeros(c.q.shape[:3], dtype=torch.bool, device="cuda")
    bad[b] = True
    assert torch.all(torch.isnan(c.o[bad])) and torch.all(torch.isnan(c.lse[bad]))
    same_elsewhere(c, o, lse, bad)


@pytest.mark.parametrize("name", sorted(FORMS))
def test_scores_of_minus_and_plus_infinity(svg, name):
    """Every key has -inf in its first channel: a row with a positive number there has scores of
    -inf alone, one with a negative number scores of +inf alone."""
    c = Case(svg, *FORMS[name], seed=23)
    c.q[..., 0] = torch.where(c.q[..., 0] < 0, -1.0, 1.0)
    c.k[..., 0] = torch.where(torch.isnan(c.k[..., 0]), c.k[..., 0], -float("inf"))
    c.call(svg)
    some, up = rows_with_keys(c), c.q[..., 0].cuda() < 0
    assert torch.all(torch.isnan(c.o[some & up])) and torch.all(torch.isnan(c.lse[some & up]))
    assert torch.all(c.o[~(some & up)] == 0) and torch.all(c.lse[~(some & up)] == -float("inf"))
