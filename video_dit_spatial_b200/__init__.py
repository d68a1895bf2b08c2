"""Python binding of libsvg, the sm_100a Sparse VideoGen sparse-attention library.

Argument marshalling only: every function here forwards to the C entry point of
the same name declared in include/svg.h (through ctypes) and raises SvgError
when it returns a non-OK status. Tensors are passed as torch tensors (their
data pointer is used), plain integer device addresses or None. All compute runs
in the library's CUDA kernels; there is no fallback. The shared library is
loaded on first use and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvg.so")

SVG_OK = 0
SVG_ERR_INVALID_ARG = 1
SVG_ERR_UNSUPPORTED = 2
SVG_ERR_CAPACITY = 3
SVG_ERR_CUDA = 4
SVG_ERR_DEVICE_TIMEOUT = 5

SVG_HEAD_SPATIAL = 0
SVG_HEAD_TEMPORAL = 1
SVG_MASK_SPATIAL = 0
SVG_MASK_TEMPORAL = 1
SVG_MASK_DENSE = 2

STATUS_NAMES = {0: "SVG_OK", 1: "SVG_ERR_INVALID_ARG", 2: "SVG_ERR_UNSUPPORTED",
                3: "SVG_ERR_CAPACITY", 4: "SVG_ERR_CUDA", 5: "SVG_ERR_DEVICE_TIMEOUT"}

EXPORTED = [
    "svg_mask_nnz", "svg_build_block_mask", "svg_profile_workspace_bytes",
    "svg_profile_heads", "svg_profile_heads_noalloc", "svg_permute", "svg_unpermute", "svg_permute_qkv",
    "svg_sparse_attention", "svg_sparse_attention_fused", "svg_quantize_v_e4m3",
    "svg_sparse_attention_fp8pv", "svg_get_device_status", "svg_selftest_wait_timeout",
    "svg2_kmeans_workspace_bytes", "svg2_kmeans", "svg2_kmeans_step", "svg2_select_clusters",
    "svg2_build_tile_csr", "svg2_gather_rows", "svg2_scatter_rows", "svg2_sparse_attention",
    "svg2_cluster_value_stats", "svg2_ear_workspace_bytes", "svg2_ear_compensate",
    "svg_cache_reset", "svg_cache_fork", "svg_cache_free", "svg_cache_reserve", "svg_cache_write",
    "svg_cache_compact", "svg_cache_copy_pages", "svg_prefix_attention_workspace_bytes",
    "svg_prefix_attention",
    "svg_status_string", "svg_version",
]


class SvgError(RuntimeError):
    def __init__(self, func: str, status: int):
        super().__init__(f"{func} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class Geom(ctypes.Structure):
    """svg_geom: geometry of one attention layer."""

    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("P", ctypes.c_int32), ("n_text", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_q", ctypes.c_int32),
                ("block_k", ctypes.c_int32), ("spatial_band", ctypes.c_int32),
                ("temporal_width", ctypes.c_int32), ("scale", ctypes.c_float)]

    @property
    def N(self) -> int:
        return self.T * self.P + self.n_text

    @property
    def n_qblocks(self) -> int:
        return -(-self.N // self.block_q)

    @property
    def n_kblocks(self) -> int:
        return -(-self.N // self.block_k)

    @classmethod
    def from_workload(cls, wl) -> "Geom":
        return cls(wl.B, wl.H, wl.T, wl.P, wl.n_text, wl.d, wl.block_q, wl.block_k,
                   wl.spatial_band, wl.temporal_width, wl.scale)


class CacheGeom(ctypes.Structure):
    """svg_cache_geom: sizes of a history cache."""

    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None

_c_geom_p = ctypes.POINTER(Geom)
_c_cache_p = ctypes.POINTER(CacheGeom)
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


def load() -> ctypes.CDLL:
    """Loads libsvg.so from the package directory (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise OSError(f"libsvg.so not found at {LIB_PATH}; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "svg_mask_nnz": [_c_geom_p, _i32, ctypes.POINTER(_i64)],
        "svg_build_block_mask": [_c_geom_p, _i32, _vp, _vp, _i64, _vp],
        "svg_profile_workspace_bytes": [_c_geom_p, _i32, ctypes.POINTER(_sz)],
        "svg_profile_heads": [_c_geom_p, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp],
        "svg_profile_heads_noalloc": [_c_geom_p, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp],
        "svg_permute": [_c_geom_p, _vp, _vp, _vp, _vp],
        "svg_unpermute": [_c_geom_p, _vp, _vp, _vp, _vp],
        "svg_permute_qkv": [_c_geom_p, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
        "svg_sparse_attention": [_c_geom_p] + [_vp] * 15,
        "svg_sparse_attention_fused": [_c_geom_p] + [_vp] * 13,
        "svg_quantize_v_e4m3": [_c_geom_p] + [_vp] * 6,
        "svg_sparse_attention_fp8pv": [_c_geom_p] + [_vp] * 15,
        "svg_get_device_status": [_vp, ctypes.POINTER(_i32)],
        "svg_selftest_wait_timeout": [_i64, _vp],
        "svg2_kmeans_workspace_bytes": [_i32, _i32, _i32, _i32, ctypes.POINTER(_sz)],
        "svg2_kmeans": [_i32, _i32, _i32, _i32, _i32] + [_vp] * 6 + [_sz, _vp],
        "svg2_kmeans_step": [_i32, _i32, _i32, _i32] + [_vp] * 7 + [_sz, _vp],
        "svg2_select_clusters": [_i32, _i32, _i32, _i32, ctypes.c_float, ctypes.c_float] +
                                [_vp] * 4 + [ctypes.c_float, _vp, _vp],
        "svg2_cluster_value_stats": [_i32] * 4 + [_vp] * 6,
        "svg2_ear_workspace_bytes": [_i32, _i32, _i32, ctypes.POINTER(_sz)],
        "svg2_ear_compensate": [_i32] * 5 + [ctypes.c_float] + [_vp] * 9 + [_sz, _vp],
        "svg2_build_tile_csr": [_i32] * 6 + [_vp] * 5 + [_i64, _vp, _vp],
        "svg2_gather_rows": [_i32, _i32, _i32, _vp, _vp, _vp, _vp],
        "svg2_scatter_rows": [_i32, _i32, _i32, _vp, _vp, _vp, _vp],
        "svg2_sparse_attention": [_i32, _i32, _i32, _i32, ctypes.c_float] + [_vp] * 8,
        "svg_cache_reset": [_c_cache_p] + [_vp] * 4,
        "svg_cache_fork": [_c_cache_p] + [_vp] * 5 + [_i32, _vp],
        "svg_cache_free": [_c_cache_p] + [_vp] * 5 + [_i32, _vp],
        "svg_cache_reserve": [_c_cache_p] + [_vp] * 5 + [_i32, _vp, _vp],
        "svg_cache_write": [_c_cache_p] + [_vp] * 3 + [_i32, _i32] + [_vp] * 5,
        "svg_cache_compact": [_c_cache_p] + [_vp] * 6,
        "svg_cache_copy_pages": [_c_cache_p, _vp, _i32] + [_vp] * 5,
        "svg_prefix_attention_workspace_bytes": [_c_cache_p, _i32, _i32, _i32,
                                                 ctypes.POINTER(_sz)],
        "svg_prefix_attention": [_c_cache_p] + [_i32] * 5 + [ctypes.c_float] + [_vp] * 9 +
                                [_sz, _vp],
        "svg_status_string": [_i32],
        "svg_version": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "svg_status_string" else ctypes.c_int32
    _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    """Device address of a buffer argument: None, a plain integer address, or a
    tensor. A tensor must live on a CUDA device and be contiguous: the kernels
    read dense row-major buffers, and a host address would fault on the device."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"libsvg takes device buffers, got a tensor on {x.device}")
    if not x.is_contiguous():
        raise ValueError("libsvg takes contiguous buffers, got a strided view")
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, status: int) -> None:
    if status != SVG_OK:
        raise SvgError(name, status)


def svg_status_string(status: int) -> str:
    return load().svg_status_string(status).decode()


def svg_version() -> int:
    return load().svg_version()


def svg_mask_nnz(geom: Geom, kind: int) -> int:
    out = _i64(0)
    _check("svg_mask_nnz", load().svg_mask_nnz(ctypes.byref(geom), kind, ctypes.byref(out)))
    return out.value


def svg_build_block_mask(geom: Geom, kind: int, row_ptr, col_idx, col_capacity=None,
                         stream=None) -> None:
    cap = col_idx.numel() if col_capacity is None else col_capacity
    _check("svg_build_block_mask", load().svg_build_block_mask(
        ctypes.byref(geom), kind, _ptr(row_ptr), _ptr(col_idx), cap, _stream(stream)))


def svg_profile_workspace_bytes(geom: Geom, n_samples: int) -> int:
    out = _sz(0)
    _check("svg_profile_workspace_bytes", load().svg_profile_workspace_bytes(
        ctypes.byref(geom), n_samples, ctypes.byref(out)))
    return out.value


def svg_profile_heads(geom: Geom, q, k, v, sample_idx, labels, mse=None, workspace=None,
                      workspace_bytes=None, n_samples=None, stream=None) -> None:
    n = sample_idx.numel() if n_samples is None else n_samples
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("svg_profile_heads", load().svg_profile_heads(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(sample_idx), n, _ptr(labels),
        _ptr(mse), _ptr(workspace), wb, _stream(stream)))


def svg_profile_heads_noalloc(geom: Geom, q, k, v, sample_idx, labels, mse=None,
                              n_samples=None, stream=None) -> None:
    """svg_profile_heads with the library's fixed internal scratch (no workspace)."""
    n = sample_idx.numel() if n_samples is None else n_samples
    _check("svg_profile_heads_noalloc", load().svg_profile_heads_noalloc(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(sample_idx), n, _ptr(labels),
        _ptr(mse), _stream(stream)))


def svg_permute(geom: Geom, inp, out, labels=None, stream=None) -> None:
    _check("svg_permute", load().svg_permute(ctypes.byref(geom), _ptr(inp), _ptr(out),
                                             _ptr(labels), _stream(stream)))


def svg_unpermute(geom: Geom, inp, out, labels=None, stream=None) -> None:
    _check("svg_unpermute", load().svg_unpermute(ctypes.byref(geom), _ptr(inp), _ptr(out),
                                                 _ptr(labels), _stream(stream)))


def svg_permute_qkv(geom: Geom, q, k, v, qp, kp, vp, labels=None, stream=None) -> None:
    _check("svg_permute_qkv", load().svg_permute_qkv(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(qp), _ptr(kp), _ptr(vp),
        _ptr(labels), _stream(stream)))


def svg_sparse_attention(geom: Geom, q, k, v, qp, kp, vp, labels, row_ptr_s, col_idx_s,
                         row_ptr_t, col_idx_t, o, op, lse=None, stream=None) -> None:
    _check("svg_sparse_attention", load().svg_sparse_attention(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(qp), _ptr(kp), _ptr(vp),
        _ptr(labels), _ptr(row_ptr_s), _ptr(col_idx_s), _ptr(row_ptr_t), _ptr(col_idx_t),
        _ptr(o), _ptr(op), _ptr(lse), _stream(stream)))


def svg_sparse_attention_fused(geom: Geom, q, k, v, kp, vp, labels, row_ptr_s, col_idx_s,
                               row_ptr_t, col_idx_t, o, lse=None, stream=None) -> None:
    _check("svg_sparse_attention_fused", load().svg_sparse_attention_fused(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(v), _ptr(kp), _ptr(vp), _ptr(labels),
        _ptr(row_ptr_s),
        _ptr(col_idx_s), _ptr(row_ptr_t), _ptr(col_idx_t), _ptr(o), _ptr(lse),
        _stream(stream)))


def svg_quantize_v_e4m3(geom: Geom, v, vp, labels, v8, v_scale, stream=None) -> None:
    _check("svg_quantize_v_e4m3", load().svg_quantize_v_e4m3(
        ctypes.byref(geom), _ptr(v), _ptr(vp), _ptr(labels), _ptr(v8), _ptr(v_scale),
        _stream(stream)))


def svg_sparse_attention_fp8pv(geom: Geom, q, k, qp, kp, v8, v_scale, labels, row_ptr_s,
                               col_idx_s, row_ptr_t, col_idx_t, o, op, lse=None,
                               stream=None) -> None:
    _check("svg_sparse_attention_fp8pv", load().svg_sparse_attention_fp8pv(
        ctypes.byref(geom), _ptr(q), _ptr(k), _ptr(qp), _ptr(kp), _ptr(v8), _ptr(v_scale),
        _ptr(labels), _ptr(row_ptr_s), _ptr(col_idx_s), _ptr(row_ptr_t), _ptr(col_idx_t),
        _ptr(o), _ptr(op), _ptr(lse), _stream(stream)))


def svg_get_device_status(stream=None):
    """(status, bits): synchronises the stream and reads/clears the device status bits."""
    bits = _i32(0)
    st = load().svg_get_device_status(_stream(stream), ctypes.byref(bits))
    return st, bits.value


def svg_selftest_wait_timeout(limit_cycles: int, stream=None) -> None:
    _check("svg_selftest_wait_timeout",
           load().svg_selftest_wait_timeout(limit_cycles, _stream(stream)))


# ---------------------------------------------------------------------------
# semantic-aware permutation (Sparse VideoGen 2)
# ---------------------------------------------------------------------------
def svg2_kmeans_workspace_bytes(BH: int, N: int, d: int, C: int) -> int:
    out = _sz(0)
    _check("svg2_kmeans_workspace_bytes",
           load().svg2_kmeans_workspace_bytes(BH, N, d, C, ctypes.byref(out)))
    return out.value


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def svg2_kmeans(BH, N, d, C, iters, x, centroids, assign, order, offsets, workspace,
                stream=None) -> None:
    _check("svg2_kmeans", load().svg2_kmeans(
        BH, N, d, C, iters, _ptr(x), _ptr(centroids), _ptr(assign), _ptr(order), _ptr(offsets),
        _ptr(workspace), _nbytes(workspace), _stream(stream)))


def svg2_kmeans_step(BH, N, d, C, x, centroids_in, centroids_out, assign, order, offsets,
                     workspace, stream=None) -> None:
    _check("svg2_kmeans_step", load().svg2_kmeans_step(
        BH, N, d, C, _ptr(x), _ptr(centroids_in), _ptr(centroids_out), _ptr(assign), _ptr(order),
        _ptr(offsets), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def svg2_select_clusters(BH, d, Cq, Ck, scale, top_p, cq, ck, offsets_k, sel, disp=None,
                         tau=0.0, stream=None) -> None:
    _check("svg2_select_clusters", load().svg2_select_clusters(
        BH, d, Cq, Ck, scale, top_p, _ptr(cq), _ptr(ck), _ptr(offsets_k), _ptr(disp), tau,
        _ptr(sel), _stream(stream)))


def svg2_cluster_value_stats(BH, N, d, Ck, v, order_k, offsets_k, vbar, disp,
                             stream=None) -> None:
    _check("svg2_cluster_value_stats", load().svg2_cluster_value_stats(
        BH, N, d, Ck, _ptr(v), _ptr(order_k), _ptr(offsets_k), _ptr(vbar), _ptr(disp),
        _stream(stream)))


def svg2_ear_workspace_bytes(BH, d, Ck) -> int:
    out = _sz(0)
    _check("svg2_ear_workspace_bytes", load().svg2_ear_workspace_bytes(BH, d, Ck,
                                                                       ctypes.byref(out)))
    return out.value


def svg2_ear_compensate(BH, N, d, Ck, block_k, scale, qs, kbar, vbar, offsets_k, row_ptr,
                        col_idx, os, lse, workspace, stream=None) -> None:
    _check("svg2_ear_compensate", load().svg2_ear_compensate(
        BH, N, d, Ck, block_k, scale, _ptr(qs), _ptr(kbar), _ptr(vbar), _ptr(offsets_k),
        _ptr(row_ptr), _ptr(col_idx), _ptr(os), _ptr(lse), _ptr(workspace), _nbytes(workspace),
        _stream(stream)))


def svg2_build_tile_csr(BH, N, Cq, Ck, block_q, block_k, offsets_q, offsets_k, sel, row_ptr,
                        col_idx, counts, col_capacity=None, stream=None) -> None:
    cap = col_idx.numel() if col_capacity is None else col_capacity
    _check("svg2_build_tile_csr", load().svg2_build_tile_csr(
        BH, N, Cq, Ck, block_q, block_k, _ptr(offsets_q), _ptr(offsets_k), _ptr(sel),
        _ptr(row_ptr), _ptr(col_idx), cap, _ptr(counts), _stream(stream)))


def svg2_gather_rows(BH, N, d, x, order, y, stream=None) -> None:
    _check("svg2_gather_rows", load().svg2_gather_rows(BH, N, d, _ptr(x), _ptr(order), _ptr(y),
                                                       _stream(stream)))


def svg2_scatter_rows(BH, N, d, y_sorted, order, y, stream=None) -> None:
    _check("svg2_scatter_rows", load().svg2_scatter_rows(BH, N, d, _ptr(y_sorted), _ptr(order),
                                                         _ptr(y), _stream(stream)))


def svg2_sparse_attention(BH, N, d, block_k, scale, qs, ks, vs, row_ptr, col_idx, os,
                          lse=None, stream=None) -> None:
    _check("svg2_sparse_attention", load().svg2_sparse_attention(
        BH, N, d, block_k, scale, _ptr(qs), _ptr(ks), _ptr(vs), _ptr(row_ptr), _ptr(col_idx),
        _ptr(os), _ptr(lse), _stream(stream)))


# ---------------------------------------------------------------------------
# history cache and the attention that reads it
# ---------------------------------------------------------------------------
_torch = None
_has_device = False


def _here():
    """torch and the current device's index, for the checks below."""
    global _torch, _has_device
    if _torch is None:
        import torch
        _has_device = torch.cuda.is_available()
        _torch = torch
    # without a device no tensor passes the checks
    return _torch, _torch.cuda.current_device() if _has_device else -2


def _buf(name: str, x, dtype, numel: int, dev: int) -> Optional[int]:
    """Device address of a buffer of the history cache: as _ptr, and a tensor
    must be on the current device, of the given type and large enough (the
    kernels take sizes from the geometry, not from the tensor)."""
    if x is None or x.__class__ is int:
        return x
    if (x.get_device() == dev and x.dtype is dtype and x.numel() >= numel and x.is_contiguous()):
        return x.data_ptr()
    _ptr(x)  # names a host tensor or a strided view
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, the current device is cuda:{dev}")
    if x.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    raise ValueError(f"{name} needs {numel} values, got {x.numel()}")


def _stream_on(dev: int, stream) -> Optional[int]:
    """As _stream; the current stream's handle without making a Stream object
    (0.1 us instead of 3 us, which is as much as the rest of a short call)."""
    if stream is None and dev >= 0:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _state(geom: CacheGeom, table, lens, refs, i32, dev: int):
    return (_buf("table", table, i32, geom.max_seqs * geom.max_pages, dev),
            _buf("lens", lens, i32, geom.max_seqs, dev),
            _buf("refs", refs, i32, geom.n_pages, dev))


def _pool_values(geom: CacheGeom) -> int:
    return geom.n_pages * geom.H_kv * geom.page_size * geom.head_dim


def svg_cache_reset(geom: CacheGeom, table, lens, refs, stream=None) -> None:
    torch, dev = _here()
    _check("svg_cache_reset", load().svg_cache_reset(
        ctypes.byref(geom), *_state(geom, table, lens, refs, torch.int32, dev),
        _stream_on(dev, stream)))


def svg_cache_fork(geom: CacheGeom, table, lens, refs, src, dst, n=None, stream=None) -> None:
    torch, dev = _here()
    i32 = torch.int32
    n = src.numel() if n is None else n
    _check("svg_cache_fork", load().svg_cache_fork(
        ctypes.byref(geom), *_state(geom, table, lens, refs, i32, dev),
        _buf("src", src, i32, n, dev), _buf("dst", dst, i32, n, dev), n, _stream_on(dev, stream)))


def svg_cache_free(geom: CacheGeom, table, lens, refs, seqs, keep=None, n=None,
                   stream=None) -> None:
    torch, dev = _here()
    i32 = torch.int32
    n = seqs.numel() if n is None else n
    _check("svg_cache_free", load().svg_cache_free(
        ctypes.byref(geom), *_state(geom, table, lens, refs, i32, dev),
        _buf("seqs", seqs, i32, n, dev), _buf("keep", keep, i32, n, dev), n,
        _stream_on(dev, stream)))


def svg_cache_reserve(geom: CacheGeom, table, lens, refs, seqs, counts, plan, n=None,
                      stream=None) -> None:
    torch, dev = _here()
    i32 = torch.int32
    n = seqs.numel() if n is None else n
    _check("svg_cache_reserve", load().svg_cache_reserve(
        ctypes.byref(geom), *_state(geom, table, lens, refs, i32, dev),
        _buf("seqs", seqs, i32, n, dev), _buf("counts", counts, i32, n, dev), n,
        _buf("plan", plan, i32, 4 * n, dev), _stream_on(dev, stream)))


def svg_cache_write(geom: CacheGeom, table, seqs, plan, L, k_new, v_new, k_pages, v_pages,
                    n=None, stream=None) -> None:
    torch, dev = _here()
    i32, bf16 = torch.int32, torch.bfloat16
    n = seqs.numel() if n is None else n
    rows, values = n * geom.H_kv * L * geom.head_dim, _pool_values(geom)
    _check("svg_cache_write", load().svg_cache_write(
        ctypes.byref(geom), _buf("table", table, i32, geom.max_seqs * geom.max_pages, dev),
        _buf("seqs", seqs, i32, n, dev), _buf("plan", plan, i32, 4 * n, dev), n, L,
        _buf("k_new", k_new, bf16, rows, dev), _buf("v_new", v_new, bf16, rows, dev),
        _buf("k_pages", k_pages, bf16, values, dev), _buf("v_pages", v_pages, bf16, values, dev),
        _stream_on(dev, stream)))


def svg_cache_compact(geom: CacheGeom, table, refs, table_out, refs_out, moves,
                      stream=None) -> None:
    torch, dev = _here()
    i32, entries = torch.int32, geom.max_seqs * geom.max_pages
    _check("svg_cache_compact", load().svg_cache_compact(
        ctypes.byref(geom), _buf("table", table, i32, entries, dev),
        _buf("refs", refs, i32, geom.n_pages, dev),
        _buf("table_out", table_out, i32, entries, dev),
        _buf("refs_out", refs_out, i32, geom.n_pages, dev),
        _buf("moves", moves, i32, 2 + 2 * geom.n_pages, dev), _stream_on(dev, stream)))


def svg_cache_copy_pages(geom: CacheGeom, moves, max_moves, k_src, v_src, k_dst, v_dst,
                         stream=None) -> None:
    torch, dev = _here()
    bf16, values = torch.bfloat16, _pool_values(geom)
    _check("svg_cache_copy_pages", load().svg_cache_copy_pages(
        ctypes.byref(geom), _buf("moves", moves, torch.int32, 2 + 2 * max_moves, dev), max_moves,
        _buf("k_src", k_src, bf16, values, dev), _buf("v_src", v_src, bf16, values, dev),
        _buf("k_dst", k_dst, bf16, values, dev), _buf("v_dst", v_dst, bf16, values, dev),
        _stream_on(dev, stream)))


def svg_prefix_attention_workspace_bytes(geom: CacheGeom, B: int, H: int, Lq: int) -> int:
    out = _sz(0)
    _check("svg_prefix_attention_workspace_bytes", load().svg_prefix_attention_workspace_bytes(
        ctypes.byref(geom), B, H, Lq, ctypes.byref(out)))
    return out.value


def svg_prefix_attention(geom: CacheGeom, B, H, Lq, prefix_seq, prefix_len, scale, q, k_pages,
                         v_pages, table, lens, seqs, o, lse, workspace, workspace_bytes=None,
                         stream=None) -> None:
    torch, dev = _here()
    i32, bf16, rows, values = torch.int32, torch.bfloat16, B * H * Lq, _pool_values(geom)
    ws, wb = workspace, workspace_bytes
    if ws is None or ws.__class__ is int:  # an address comes with its size
        wb = 0 if wb is None else wb
    else:
        ws, wb = _buf("workspace", ws, ws.dtype, 0, dev), _nbytes(ws) if wb is None else wb
    _check("svg_prefix_attention", load().svg_prefix_attention(
        ctypes.byref(geom), B, H, Lq, prefix_seq, prefix_len, scale,
        _buf("q", q, bf16, rows * geom.head_dim, dev),
        _buf("k_pages", k_pages, bf16, values, dev), _buf("v_pages", v_pages, bf16, values, dev),
        _buf("table", table, i32, geom.max_seqs * geom.max_pages, dev),
        _buf("lens", lens, i32, geom.max_seqs, dev), _buf("seqs", seqs, i32, B, dev),
        _buf("o", o, bf16, rows * geom.head_dim, dev), _buf("lse", lse, torch.float32, rows, dev),
        ws, wb, _stream_on(dev, stream)))
