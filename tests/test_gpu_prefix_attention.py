"""GPU parity of svg_prefix_attention against the fp64 oracle, and a run of the
history cache with it as a generator uses them.

Tolerance, element by element. The kernel's only roundings to 16 bits are the
weights it feeds to the tensor core (each off by at most 2^-8 of itself, half a
bf16 step) and the output (2^-8 of itself). The first moves O by at most
2^-8 sum_j w_j |v_j|, which the oracle gives as `spread`. In 32 bits: a logit is off by a
few 2^-24 of sum |q_i k_i| scale <= 2^-20 X with X the largest |q| |k| scale of
the case, which moves every weight by that much relative to itself; sums of n
terms by less than 2^-20. So
    |O - O*| <= (2^-8 + 2^-19 (1 + X)) spread + 2^-8 |O*| + 2^-8 times the first term,
    |lse - lse*| <= 2^-19 (1 + X) + 2^-22 |lse*|.
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import cache_oracle as CO
from gpu_util import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svg():
    import video_dit_spatial_b200 as m
    m.load()
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A pool with scattered pages: sequence 0 is the history, the others share
    its whole pages and have their own rows after `prefix`. Every row that no
    sequence has holds NaN."""

    def __init__(self, svg, B, H, H_kv, d, ps, prefix, Lq, tails, seed=0, idle=(), q_scale=1.0,
                 spare_seqs=1):
        rng = np.random.default_rng(seed)
        self.B, self.H, self.Lq, self.prefix, self.ps = B, H, Lq, prefix, ps
        shared, full = -(-prefix // ps), prefix // ps
        lens = [prefix] + [prefix + t for t in tails] + [0] * spare_seqs
        n_own = [-(-(prefix + t) // ps) - full if t else 0 for t in tails]
        n_pages = shared + sum(n_own) + 2
        ids = rng.permutation(n_pages)
        width = max([1, shared] + [full + n for n in n_own]) + 1
        table = np.full((len(lens), width), -1, dtype=np.int32)
        table[0, :shared] = ids[:shared]
        at = shared
        for b, n in enumerate(n_own):
            table[b + 1, :full] = ids[:full]
            table[b + 1, full:full + n] = ids[at:at + n]
            at += n
            if not n and shared > full:
                table[b + 1, full] = ids[full]
        g = torch.Generator().manual_seed(seed)
        shape = (n_pages, H_kv, ps, d)
        pools = []
        for _ in range(2):
            x = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            val = torch.randn(shape, generator=g).to(torch.bfloat16)
            for s, n in enumerate(lens):
                for slot in range(-(-n // ps)):
                    rows = min(ps, n - slot * ps)
                    page = int(table[s, slot])
                    x[page, :, :rows] = val[page, :, :rows]
            if prefix % ps:  # the copies of the history's open page
                for b, n in enumerate(n_own):
                    if n:
                        x[int(table[b + 1, full]), :, :prefix % ps] = \
                            x[int(table[0, full]), :, :prefix % ps]
            pools.append(x)
        self.q = (q_scale * torch.randn((B, H, Lq, d), generator=g)).to(torch.bfloat16)
        self.k, self.v = pools
        self.scale = float(np.float32(d ** -0.5))
        self.table, self.lens = table, lens
        self.seqs = [-1 if b in idle else b + 1 for b in range(B)]
        self.prefix_seq = 0
        self.geom = svg.CacheGeom(n_pages, ps, H_kv, d, len(lens), width)

    def call(self, svg, o=None, lse=None, stream=None, with_lse=True):
        B, H, Lq, d = self.q.shape
        self.dq, self.dk, self.dv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.o = torch.full((B, H, Lq, d), 7.5, dtype=torch.bfloat16, device="cuda") if o is None else o
        self.lse = torch.full((B, H, Lq), 7.5, device="cuda") if with_lse else None
        self.args = (self.geom, B, H, Lq, self.prefix_seq, self.prefix, self.scale, self.dq,
                     self.dk, self.dv, dev(self.table), dev(self.lens), dev(self.seqs), self.o,
                     self.lse)
        need = svg.svg_prefix_attention_workspace_bytes(self.geom, B, H, Lq)
        self.ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read
        svg.svg_prefix_attention(*self.args, self.ws)
        st, bits = svg.svg_get_device_status()
        assert st == svg.SVG_OK and bits == 0, (st, bits)
        return self

    def compare(self, what=""):
        qn, kn, vn = to_f64(self.q), to_f64(self.k), to_f64(self.v)
        want, wlse, spread = CO.prefix_attention(qn, kn, vn, self.table, self.lens, self.seqs,
                                                 self.prefix_seq, self.prefix, self.scale, self.ps)
        got = to_f64(self.o)
        busy = np.array([s >= 0 for s in self.seqs])
        assert np.all(got[~busy] == 7.5)
        got, want, wlse, spread = got[busy], want[busy], wlse[busy], spread[busy]
        kmax = np.sqrt(np.nanmax(np.sum(kn * kn, axis=-1), initial=0.0))
        X = np.sqrt(np.max(np.sum(qn * qn, axis=-1))) * kmax * self.scale
        soft = 2.0 ** -8 + 2.0 ** -19 * (1.0 + X)
        tol = soft * spread * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        assert np.all(np.isfinite(got)), what
        err = np.abs(got - want)
        assert np.all(err <= tol), (what, float(np.max(err - tol)))
        n = np.sqrt(np.sum(want * want))
        if n > 0:
            assert np.sqrt(np.sum(err * err)) <= 1e-2 * n
        if self.lse is not None:
            gl = self.lse.cpu().numpy().astype(np.float64)
            assert np.all(gl[~busy] == 7.5)
            gl = gl[busy]
            none = np.isneginf(wlse)
            assert np.array_equal(np.isneginf(gl), none)
            assert np.all(np.abs(gl[~none] - wlse[~none]) <=
                          2.0 ** -19 * (1 + X) + 2.0 ** -22 * np.abs(wlse[~none]))


# B, H, H_kv, d, page, prefix, Lq, tails
CASES = {
    "one_key": (1, 1, 1, 64, 16, 1, 1, [0]),
    "one_key_of_its_own": (1, 1, 1, 128, 16, 0, 1, [1]),
    "nothing_shared": (3, 4, 2, 64, 16, 0, 1, [5, 0, 130]),
    "no_rows_at_all": (2, 2, 1, 128, 32, 0, 3, [0, 0]),
    "only_the_prefix": (4, 2, 2, 128, 64, 128, 1, [0, 0, 0, 0]),
    "ends_with_a_page": (3, 3, 3, 64, 16, 160, 1, [1, 16, 17]),
    "ends_inside_a_page": (5, 4, 1, 128, 32, 333, 1, [1, 2, 90, 0, 300]),
    "page_256": (3, 4, 2, 64, 256, 700, 2, [2, 70, 600]),
    "page_128": (2, 6, 2, 128, 128, 1025, 3, [3, 127]),
    "one_row_long": (2, 2, 2, 128, 64, 9001, 1, [33, 200]),
    "grouped": (9, 16, 2, 128, 16, 500, 1, list(range(0, 270, 30))),
    "many_rows_each": (2, 4, 2, 64, 16, 300, 150, [150, 200]),
    "rows_127": (2, 1, 1, 128, 64, 257, 127, [127, 129]),
    "rows_128": (2, 1, 1, 128, 64, 256, 128, [128, 128]),
    "rows_129": (2, 1, 1, 64, 64, 255, 129, [0, 1000]),
    "rows_256": (1, 2, 2, 128, 128, 640, 256, [256]),
    "rows_257": (3, 2, 1, 64, 32, 100, 257, [257, 300, 0]),
    "rows_700": (2, 2, 2, 128, 16, 900, 700, [700, 5]),
    "tiles_cross_sequences": (7, 6, 2, 64, 16, 411, 31, [31, 40, 0, 1, 500, 128, 127]),
    "long_tails": (2, 2, 1, 64, 16, 16, 1, [5000, 3]),
    "batch_300": (300, 2, 1, 64, 16, 200, 1, [i % 41 for i in range(300)]),
    "batch_1024": (1024, 1, 1, 64, 16, 33, 1, [i % 3 for i in range(1024)]),
    "one_sequence": (1, 8, 2, 128, 64, 1000, 5, [5]),
    "heads_40": (2, 40, 40, 64, 16, 90, 1, [3, 20]),
    # warps without rows beside warps with them, over many blocks
    "second_tile_of_few_rows": (36, 8, 2, 64, 32, 5000, 1, [i % 50 for i in range(36)]),
    "one_tile_of_some_rows": (60, 16, 16, 64, 128, 300, 1, [900 + 7 * i for i in range(60)]),
    # several long items to every CTA
    "long_tails_of_many": (12, 24, 24, 64, 64, 300, 1, [900 + 97 * i for i in range(12)]),
    "long_tails_of_rows": (12, 24, 12, 128, 128, 700, 20, [600 + 97 * i for i in range(12)]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_parity(svg, name):
    Case(svg, *CASES[name], seed=sorted(CASES).index(name)).call(svg).compare(name)


# More items than SMs, so that each SM has whole ones before its piece of the rest: of one
# sequence each, with a prefix and without, of all sequences together, and beside the
# kernel for few rows. Some sequences have no rows of their own.
DEALT = {
    "own_and_prefix": (3, 40, 40, 64, 64, 600, 900, [900, 0, 1400]),
    "own": (6, 24, 24, 128, 16, 0, 260, [700, 690, 0, 701, 640, 768]),
    "gathered": (30, 60, 60, 64, 32, 700, 20, [7 * b for b in range(30)]),
    "gathered_long": (5, 80, 80, 128, 128, 2000, 60, [60, 0, 200, 61, 1000]),
    "beside_few_rows": (150, 240, 60, 64, 16, 1000, 1, [b % 60 for b in range(150)]),
}


@pytest.mark.parametrize("name", sorted(DEALT))
@pytest.mark.parametrize("idle", [(), (1,)])
def test_more_items_than_sms(svg, name, idle):
    Case(svg, *DEALT[name], seed=17, idle=idle).call(svg).compare(name)


@pytest.mark.parametrize("d,H,H_kv,Lq", [(64, 160, 160, 17), (128, 4, 2, 200), (128, 8, 4, 1),
                                         (64, 200, 200, 1)])
def test_the_longest_table(svg, d, H, H_kv, Lq):
    """2^20 rows, the same seven pages over and over: the answer is that of one round of them
    and the sum 585 times as large. Sums of one sign at a time are where rounding adds up: O
    takes 16 keys at a time, 2^16 sums that lose up to 2^-24 each, so 2^-8 of `spread`; the
    row sum 2^14 of them (a key pair at a time within a block, then block by block), 2^-10."""
    ps, n_pages = 256, 7
    W = (1 << 20) // ps
    rounds = W // n_pages
    n = rounds * n_pages * ps
    g = torch.Generator().manual_seed(d + H)
    k, v = (torch.randn((n_pages, H_kv, ps, d), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, H, Lq, d), generator=g).to(torch.bfloat16)
    table = (torch.arange(W, dtype=torch.int32) % n_pages).repeat(2, 1)
    geom = svg.CacheGeom(n_pages, ps, H_kv, d, 2, W)
    o = torch.empty((1, H, Lq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, H, Lq), device="cuda")
    ws = torch.empty(svg.svg_prefix_attention_workspace_bytes(geom, 1, H, Lq), dtype=torch.uint8,
                     device="cuda")
    svg.svg_prefix_attention(geom, 1, H, Lq, 0, n, d ** -0.5, q.cuda(), k.cuda(), v.cuda(),
                             table.cuda(), dev([n, n]), dev([1]), o, lse, ws)
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)
    kk, vv = (x.transpose(0, 1).reshape(H_kv, -1, d).repeat_interleave(H // H_kv, 0).double()
              for x in (k, v))
    z = q[0].double() @ kk.transpose(1, 2) * float(np.float32(d ** -0.5))
    w = torch.softmax(z, -1)
    want, spread = w @ vv, w @ vv.abs()
    want_lse = torch.logsumexp(z, -1) + np.log(rounds)
    X = float(q.double().norm(dim=-1).max() * kk.norm(dim=-1).max()) * d ** -0.5
    soft = 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -19 * (1 + X)
    assert torch.all((o[0].cpu().double() - want).abs() <=
                     soft * spread * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs())
    assert torch.all((lse[0].cpu().double() - want_lse).abs() <=
                     2.0 ** -10 + 2.0 ** -19 * (1 + X) + 2.0 ** -22 * want_lse.abs())


@pytest.mark.parametrize("name", ["grouped", "tiles_cross_sequences", "rows_257"])
def test_idle_entries_keep_their_rows(svg, name):
    a = CASES[name]
    Case(svg, *a, seed=5, idle=(0, a[0] - 1)).call(svg).compare(name)
    c = Case(svg, *a, seed=5, idle=range(a[0])).call(svg)
    assert torch.all(c.o == 7.5) and torch.all(c.lse == 7.5)


@pytest.mark.parametrize("name", ["ends_inside_a_page", "many_rows_each", "rows_700"])
def test_peaked_rows(svg, name):
    """Logits far apart: the running maximum moves by hundreds."""
    Case(svg, *CASES[name], seed=6, q_scale=60.0).call(svg).compare(name)


def test_without_lse(svg):
    c = Case(svg, *CASES["grouped"], seed=7).call(svg)
    o = c.o.clone()
    c.call(svg, with_lse=False)
    assert torch.equal(o, c.o)


def test_the_same_sequence_twice_and_a_prefix_of_the_batch(svg):
    c = Case(svg, 4, 4, 2, 64, 16, 200, 2, [20, 7, 50, 9], seed=8)
    c.seqs = [2, 3, 2, 1]
    c.prefix_seq = 3  # holds the same rows
    c.call(svg).compare()


def test_a_prefix_shorter_than_what_is_shared(svg):
    """The caller may name fewer shared rows than the sequences have in common."""
    c = Case(svg, 3, 2, 2, 128, 32, 300, 1, [20, 7, 50], seed=9)
    c.prefix = 250
    c.call(svg).compare()
    c.prefix = 0
    c.call(svg).compare()


def test_a_sequence_shorter_than_the_prefix_sees_the_prefix_alone(svg):
    c = Case(svg, 3, 2, 2, 128, 32, 300, 1, [20, 7, 50], seed=10)
    c.lens[2] = 100
    c.call(svg).compare()


def test_equal_results_on_every_call(svg):
    for name in ("grouped", "one_row_long", "rows_700", "second_tile_of_few_rows",
                 "one_tile_of_some_rows", "rows_129"):
        c = Case(svg, *CASES[name], seed=11).call(svg)
        o, lse = c.o.clone(), c.lse.clone()
        for _ in range(20):
            c.o.fill_(1.0)
            svg.svg_prefix_attention(*c.args, c.ws)
            assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_large_inputs_keep_to_their_rows(svg):
    """A sequence whose keys and values are infinite or NaN does not reach the others."""
    c = Case(svg, 4, 4, 2, 64, 16, 100, 3, [20, 30, 40, 50], seed=12).call(svg)
    o = c.o.clone()
    bad = int(c.table[2, 8])  # a page of its own of the second entry
    for x, y in ((float("inf"), float("nan")), (float("nan"), float("-inf"))):
        c.k[bad], c.v[bad] = x, y
        c.call(svg)
        assert torch.equal(c.o[[0, 2, 3]], o[[0, 2, 3]])


def test_flagged_sequences_are_left_out(svg):
    c = Case(svg, 4, 4, 2, 64, 16, 100, 3, [20, 30, 40, 50], seed=13).call(svg)
    o, lse = c.o.clone(), c.lse.clone()
    seqs, lens = dev([1, 99, 3, 4]), dev(c.lens)
    lens[3] = 16 * c.geom.max_pages + 1
    args = list(c.args)
    args[11], args[12] = lens, seqs
    c.o.fill_(3.0)
    c.lse.fill_(3.0)
    svg.svg_prefix_attention(*args, c.ws)
    assert svg.svg_get_device_status()[1] == 2
    assert torch.equal(c.o[[0, 3]], o[[0, 3]]) and torch.equal(c.lse[[0, 3]], lse[[0, 3]])
    assert torch.all(c.o[[1, 2]] == 3.0) and torch.all(c.lse[[1, 2]] == 3.0)
    lens[0] = 99  # the history is shorter than the prefix
    c.o.fill_(3.0)
    svg.svg_prefix_attention(*args, c.ws)
    assert svg.svg_get_device_status()[1] == 2
    assert torch.all(c.o == 3.0)


@pytest.mark.parametrize("name", ["tiles_cross_sequences", "page_256", "rows_700"])
def test_a_page_past_the_pool_counts_as_zeros(svg, name):
    c = Case(svg, *CASES[name], seed=14)
    slot, own = 1, c.prefix // c.ps + 1
    c.k[c.table[0, slot]] = 0.0
    c.v[c.table[0, slot]] = 0.0
    c.k[c.table[2, own]] = 0.0
    c.v[c.table[2, own]] = 0.0
    c.call(svg).compare()
    o = c.o.clone()
    args = list(c.args)
    table = dev(c.table)
    table[0, slot], table[2, own] = c.geom.n_pages, -5
    args[10] = table
    svg.svg_prefix_attention(*args, c.ws)
    assert svg.svg_get_device_status()[1] == 2
    assert torch.equal(c.o, o)


def test_streams_and_replayed_graphs(svg):
    """Two streams with workspaces of their own, and a captured call replayed on new inputs."""
    a = Case(svg, *CASES["grouped"], seed=15).call(svg)
    b = Case(svg, *CASES["rows_700"], seed=16).call(svg)
    oa, ob = a.o.clone(), b.o.clone()
    a.o.zero_(), b.o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for c, s in zip((a, b), streams):
            svg.svg_prefix_attention(*c.args, c.ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.o, oa) and torch.equal(b.o, ob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svg.svg_prefix_attention(*a.args, a.ws)
    other = Case(svg, *CASES["grouped"], seed=17).call(svg)
    a.dq.copy_(other.dq)
    a.dk.copy_(other.dk)
    a.dv.copy_(other.dv)
    a.args[10].copy_(other.args[10])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o, other.o) and torch.equal(a.lse, other.lse)


def test_binding_refuses_what_does_not_fit(svg):
    c = Case(svg, *CASES["grouped"], seed=18).call(svg)
    for at, bad in ((7, c.dq.float()), (7, c.dq[:1]), (7, torch.stack([c.dq] * 2, -1)[..., 0]), (8, c.dk[:-1]),
                    (10, c.args[10].long()), (11, c.args[11][:1]), (14, c.lse.double())):
        args = list(c.args)
        args[at] = bad
        with pytest.raises(ValueError):
            svg.svg_prefix_attention(*args, c.ws)
    with pytest.raises(svg.SvgError) as e:
        svg.svg_prefix_attention(*c.args, c.ws, workspace_bytes=8)
    assert e.value.status == svg.SVG_ERR_CAPACITY


@pytest.mark.parametrize("ps,d,H,H_kv", [(16, 64, 4, 2), (64, 128, 3, 3)])
def test_chunk_by_chunk(svg, ps, d, H, H_kv):
    """Two layers, a history of two frames, three continuations of two frames
    each; one is dropped, another cut back and taken up again, the pools
    compacted. Every attention against fp64 over the rows that went in."""
    from video_dit_spatial_b200.layer import HistoryCache
    P, layers = 75, 2
    cache = HistoryCache(layers, 60 if ps == 16 else 24, ps, H, H_kv, d, max_seqs=6, max_rows=5 * P,
                         batch=3, rows=P)
    g = torch.Generator().manual_seed(ps)
    rows = {s: [[[], []] for _ in range(layers)] for s in range(6)}  # per sequence and layer: K, V parts

    def rand(n, heads, L):
        return torch.randn((n, heads, L, d), generator=g).to(torch.bfloat16)

    def chunk(seqs, prefix_len, L=P):
        s = dev(seqs)
        cache.reserve(s, dev([L] * len(seqs)))
        q, o = rand(len(seqs), H, L).cuda(), torch.empty((len(seqs), H, L, d), dtype=torch.bfloat16,
                                                         device="cuda")
        for layer in range(layers):
            for step in range(2):  # the chunk's rows are written again at the second step
                k, v = rand(len(seqs), H_kv, L), rand(len(seqs), H_kv, L)
                cache.write(layer, k.cuda(), v.cuda())
            for i, x in enumerate(seqs):
                rows[x][layer][0].append(k[i])
                rows[x][layer][1].append(v[i])
            cache.attend(layer, q, s, seqs[0], prefix_len, o)
            assert svg.svg_get_device_status()[1] == 0
            for i, x in enumerate(seqs):
                kk, vv = (to_f64(torch.cat(y, dim=1)) for y in rows[x][layer])
                qn = to_f64(q[i])
                for h in range(H):
                    z = qn[h] @ kk[h // (H // H_kv)].T * d ** -0.5
                    w = np.exp(z - z.max(axis=1, keepdims=True))
                    w /= w.sum(axis=1, keepdims=True)
                    vh = vv[h // (H // H_kv)]
                    want = w @ vh
                    X = np.abs(z).max() * 16
                    tol = (2.0 ** -8 + 2.0 ** -19 * (1 + X)) * (w @ np.abs(vh)) * (1 + 2.0 ** -8) + \
                        2.0 ** -8 * np.abs(want)
                    assert np.all(np.abs(to_f64(o[i, h]) - want) <= tol)

    def fork(src, dst):
        cache.fork(dev(src), dev(dst))
        for s, t in zip(src, dst):
            rows[t] = [[list(part) for part in layer] for layer in rows[s]]

    chunk([0], 0)
    chunk([0], P)
    fork([0, 0, 0], [1, 2, 3])
    chunk([1, 2, 3], 2 * P)
    cache.free(dev([2]))
    cache.compact()
    with pytest.raises(ValueError):
        cache.write(0, rand(3, H_kv, P).cuda(), rand(3, H_kv, P).cuda())
    chunk([3, 1], 2 * P)
    cache.free(dev([3, 0]), dev([3 * P, 0]))
    for layer in rows[3]:
        for part in layer:
            part.pop()
    fork([3], [4])
    cache.compact()
    chunk([4, 3], 3 * P, L=P - 20)
