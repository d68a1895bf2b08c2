"""HistoryCache without a GPU: what it gives to the calls below it, which are recorded."""
import pytest
import torch

import video_dit_spatial_b200 as svg
from video_dit_spatial_b200.layer import HistoryCache

CALLS = ("svg_cache_reset", "svg_cache_fork", "svg_cache_free", "svg_cache_reserve",
         "svg_cache_write", "svg_cache_compact", "svg_cache_copy_pages", "svg_prefix_attention")


@pytest.fixture()
def calls(monkeypatch):
    """The calls made, in order: (name, copies of the tensors among the arguments, keywords)."""
    made = []

    def record(name):
        def call(*args, **kw):
            made.append((name, [x.clone() if torch.is_tensor(x) else x for x in args], kw))
        return call

    for name in CALLS:
        monkeypatch.setattr(svg, name, record(name))
    monkeypatch.setattr(svg, "svg_prefix_attention_workspace_bytes", lambda *a: 256)
    return made


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def test_write_names_the_sequences_that_reserve_was_given(calls):
    cache = HistoryCache(2, 8, 16, 2, 1, 64, 6, 64, 3, 8, device="cpu")
    seqs, rows = ints([0, 4]), torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16)
    cache.reserve(seqs, ints([8, 3]))
    seqs.copy_(ints([2, 3]))
    cache.write(0, rows, rows)
    del seqs
    cache.write(1, rows, rows)
    assert [args[2][:kw["n"]].tolist() for name, args, kw in calls if name == "svg_cache_write"] == \
        [[0, 4]] * 2
    cache.reserve(ints([1]), ints([1]))
    with pytest.raises(ValueError, match="rows of shape"):
        cache.write(0, rows, rows)
    cache.fork(ints([0]), ints([5]))
    with pytest.raises(ValueError, match="follows reserve"):
        cache.write(0, rows[:1], rows[:1])


def test_check_raises_what_the_device_refused(calls, monkeypatch):
    cache = HistoryCache(1, 8, 16, 2, 1, 64, 6, 64, 3, 8, device="cpu")
    for status in (svg.SVG_ERR_CAPACITY, svg.SVG_ERR_INVALID_ARG, svg.SVG_ERR_DEVICE_TIMEOUT,
                   svg.SVG_ERR_CUDA):
        monkeypatch.setattr(svg, "svg_get_device_status", lambda stream: (status, 0))
        with pytest.raises(svg.SvgError) as e:
            cache.check()
        assert e.value.status == status
    monkeypatch.setattr(svg, "svg_get_device_status", lambda stream: (svg.SVG_OK, stream))
    cache.check(stream=7)


def test_attention_without_a_workspace_is_a_status():
    """As every other null, and as an address whose size is not given."""
    from video_dit_spatial_b200 import _build
    _build.build()
    geom = svg.CacheGeom(8, 16, 2, 64, 4, 5)
    for workspace, size, status in ((None, None, svg.SVG_ERR_INVALID_ARG),
                                    (None, 1 << 30, svg.SVG_ERR_INVALID_ARG),
                                    (256, None, svg.SVG_ERR_CAPACITY),
                                    (256, 64, svg.SVG_ERR_CAPACITY)):
        with pytest.raises(svg.SvgError) as e:
            svg.svg_prefix_attention(geom, 2, 4, 3, 0, 17, 0.1, 1 << 20, 256, 256, 256, 256, 256, 256,
                                     None, workspace, workspace_bytes=size)
        assert e.value.status == status


def test_a_device_that_is_not_current_is_refused_before_anything_is_allocated(calls, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def no(*a, **kw):
        raise AssertionError("allocated")

    monkeypatch.setattr(torch, "empty", no)
    with pytest.raises(ValueError, match="make cuda:1 the current one"):
        HistoryCache(1, 8, 16, 2, 1, 64, 6, 64, 3, 8, device="cuda:1")
    for device in ("cuda", "cuda:0"):
        with pytest.raises(AssertionError, match="allocated"):
            HistoryCache(1, 8, 16, 2, 1, 64, 6, 64, 3, 8, device=device)
