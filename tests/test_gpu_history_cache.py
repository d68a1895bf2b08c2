"""HistoryCache: what its calls keep, and what it says of a refusal."""
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


def rows(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def rows_of(cache, layer, seq, lo, hi):
    """Keys and values at positions [lo, hi) of a sequence: [H_kv, hi - lo, d] each."""
    ps, entries = cache.geom.page_size, cache.table[seq].tolist()
    at = range(lo, hi)
    return [torch.stack([x[entries[p // ps], :, p % ps] for p in at], 1)
            for x in cache.pools[layer]]


@pytest.mark.parametrize("named", ["current", "stream", "handle", "handle of the default stream"])
def test_a_list_refilled_after_reserve(svg, named):
    """One buffer for the batch's numbers, refilled before the last layer is written: the
    rows still go to the sequences that reserve made room for."""
    from video_dit_spatial_b200.layer import HistoryCache
    cache = HistoryCache(2, 16, 16, 2, 2, 64, 6, 64, 3, 8)
    seqs = dev([0, 4, 1])
    side = torch.cuda.default_stream() if "default" in named else torch.cuda.Stream()
    on = {"current": None, "stream": side}.get(named, side.cuda_stream)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        k, v, others = rows(3, 2, 8, 64), rows(3, 2, 8, 64), dev([2, 3, 5])
        full, counts = dev([20, 20, 20]), dev([8, 8, 5])
        side.synchronize()
        with torch.cuda.stream(side if on is None else torch.cuda.Stream()):
            cache.reserve(others, full, stream=on)
            cache.reserve(seqs, counts, stream=on)
        before = [[x.clone() for x in pool] for pool in cache.pools]
        cache.write(0, k, v, stream=on)
        seqs.copy_(dev([2, 3, -1]))
        cache.write(1, k, v, stream=on)
        for layer in range(2):
            for i, (s, n) in enumerate(((0, 8), (4, 8), (1, 5))):
                for got, want in zip(rows_of(cache, layer, s, 0, n), (k[i, :, :n], v[i, :, :n])):
                    assert torch.equal(got, want)
            pages = [p for s in (2, 3, 5) for p in cache.table[s, :2].tolist()]
            for x, y in zip(cache.pools[layer], before[layer]):
                assert torch.equal(x[pages].view(torch.int16), y[pages].view(torch.int16))
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)


def test_a_captured_step_takes_the_list_as_it_is_replayed(svg):
    from video_dit_spatial_b200.layer import HistoryCache
    cache = HistoryCache(1, 16, 16, 2, 2, 64, 6, 64, 2, 8)
    seqs, counts, k, v = dev([0, 1]), dev([8, 3]), rows(2, 2, 8, 64), rows(2, 2, 8, 64)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.reserve(seqs, counts)
        cache.write(0, k, v)
    for numbers in ([0, 1], [4, -1], [1, 0]):
        lens = cache.lens.tolist()
        seqs.copy_(dev(numbers))
        graph.replay()
        for i, (s, n) in enumerate(zip(numbers, (8, 3))):
            if s >= 0:
                got = rows_of(cache, 0, s, lens[s], lens[s] + n)
                assert torch.equal(got[0], k[i, :, :n]) and torch.equal(got[1], v[i, :, :n])
    assert cache.lens.tolist() == [11, 11, 0, 0, 8, 0]
    assert svg.svg_get_device_status() == (svg.SVG_OK, 0)


def test_a_full_pool_is_told_by_check(svg):
    """Without room nothing is reserved or written, and attend reads the rows that were there."""
    from video_dit_spatial_b200.layer import HistoryCache
    cache = HistoryCache(1, 4, 16, 2, 2, 64, 3, 128, 2, 16)
    k, v = rows(2, 2, 16, 64), rows(2, 2, 16, 64)
    seqs, q, o = dev([0, 1]), rows(2, 2, 16, 64), rows(2, 2, 16, 64)
    cache.reserve(seqs, dev([16, 16]))
    cache.check()
    cache.write(0, k, v)
    cache.attend(0, q, seqs, 0, 0, o)
    want = o.clone()
    held = [[x.clone() for x in pool] for pool in cache.pools] + [[x.clone() for x in cache._state]]
    cache.reserve(seqs, dev([16, 17]))  # three pages of two
    cache.write(0, v, k)
    cache.attend(0, q, seqs, 0, 0, o)
    with pytest.raises(svg.SvgError) as e:
        cache.check()
    assert e.value.status == svg.SVG_ERR_CAPACITY
    cache.check()  # told once
    for now, before in zip(cache.pools + [cache._state], held):
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(now, before))
    assert torch.equal(o, want)
    cache.reserve(seqs, dev([16, 16]))
    cache.check()
    cache.fork(dev([0]), dev([9]))
    with pytest.raises(svg.SvgError) as e:
        cache.check()
    assert e.value.status == svg.SVG_ERR_INVALID_ARG


def test_a_stream_of_another_kind(svg):
    """Whatever has a cuda_stream, as in every other call."""
    from video_dit_spatial_b200.layer import HistoryCache

    class Other:
        cuda_stream = torch.cuda.Stream().cuda_stream

    cache = HistoryCache(1, 16, 16, 2, 2, 64, 6, 64, 3, 8)
    seqs, counts, k, v = dev([4, 1]), dev([8, 5]), rows(2, 2, 8, 64), rows(2, 2, 8, 64)
    torch.cuda.synchronize()
    cache.reserve(seqs, counts, stream=Other)
    cache.write(0, k, v, stream=Other)
    cache.check(stream=Other)
    for i, (s, n) in enumerate(((4, 8), (1, 5))):
        assert all(torch.equal(x, y[i, :, :n]) for x, y in zip(rows_of(cache, 0, s, 0, n), (k, v)))
