"""One Sparse VideoGen attention layer on the GPU: buffers plus the call sequence.

The path (arXiv 2502.01776, abstract): online profiling labels every head
spatial or temporal; temporal heads are moved to position-major order (the
layout transformation); block-sparse attention runs over each head's block
mask; temporal outputs are moved back. This class only owns device buffers
(allocated with torch) and calls the library's entry points in that order on
one stream; every step is a libsvg kernel.

`layout` chooses how the layout transformation is done:
  "explicit"  permute Q, K, V of temporal heads, attend, un-permute O (the
              default: the fastest);
  "fused"     permute K, V only; the attention kernel gathers the query rows of
              temporal heads in position-major order and stores each output row
              at its frame-major place (no Q or O copies, no un-permute pass;
              about 1 % slower, since the row gathers cost about what the
              dropped passes save);
  "gathered"  nothing is permuted: key/value rows are gathered in the kernel
              too (least memory; far slower, row gathers move fewer bytes per
              cycle than tiled loads).
"fused" and "gathered" need 128-row query blocks; they give the same bits as
"explicit".

`pv` chooses the arithmetic of the PV product: "bf16" (the default) or
"e4m3" (FP8: V quantised per (head, channel) by svg_quantize_v_e4m3, P
rounded to e4m3 inside the kernel; explicit layout, d = 128, 128-row query
blocks only; a looser tolerance than bf16).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (Geom, SVG_MASK_DENSE, SVG_MASK_SPATIAL, SVG_MASK_TEMPORAL, _stream, svg_build_block_mask,
               svg_mask_nnz, svg_permute_qkv, svg_profile_heads, svg_profile_workspace_bytes,
               svg_quantize_v_e4m3, svg_sparse_attention, svg_sparse_attention_fp8pv,
               svg_sparse_attention_fused, svg_unpermute)


class BlockMaskCSR:
    """Device CSR of one block mask (built once per geometry)."""

    def __init__(self, geom: Geom, kind: int, device):
        self.kind = kind
        self.nnz = svg_mask_nnz(geom, kind)
        self.row_ptr = torch.empty(geom.n_qblocks + 1, dtype=torch.int32, device=device)
        self.col_idx = torch.empty(max(self.nnz, 1), dtype=torch.int32, device=device)

    def build(self, geom: Geom, stream=None) -> None:
        svg_build_block_mask(geom, self.kind, self.row_ptr, self.col_idx, stream=stream)


LAYOUTS = ("explicit", "fused", "gathered")


class SparseVideoGenLayer:
    def __init__(self, geom: Geom, n_samples: int, device="cuda",
                 layout: Optional[str] = None, pv: str = "bf16"):
        self.geom = geom
        if layout is None:
            layout = "explicit"
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {LAYOUTS}")
        if pv not in ("bf16", "e4m3"):
            raise ValueError("pv must be 'bf16' or 'e4m3'")
        if pv == "e4m3" and layout != "explicit":
            raise ValueError("the e4m3 PV product runs on the explicit layout")
        self.layout = layout
        self.pv = pv
        self.n_samples = n_samples
        self.device = torch.device(device)
        B, H, N, d = geom.B, geom.H, geom.N, geom.head_dim
        shape = (B, H, N, d)
        self.masks = {k: BlockMaskCSR(geom, k, self.device)
                      for k in (SVG_MASK_SPATIAL, SVG_MASK_TEMPORAL)}
        self.dense_mask: Optional[BlockMaskCSR] = None
        wbytes = svg_profile_workspace_bytes(geom, n_samples)
        self.workspace = torch.empty(max(wbytes // 4, 1), dtype=torch.float32, device=self.device)
        self.labels = torch.empty(B * H, dtype=torch.int8, device=self.device)
        self.mse = torch.empty(B * H * 2, dtype=torch.float32, device=self.device)
        self.qp = self.kp = self.vp = self.op = None
        mk = lambda: torch.empty(shape, dtype=torch.bfloat16, device=self.device)  # noqa: E731
        if layout == "explicit":
            self.qp, self.op = mk(), mk()
        if layout in ("explicit", "fused"):
            self.kp, self.vp = mk(), mk()
        self.v8 = self.v_scale = None
        if pv == "e4m3":
            self.v8 = torch.empty(shape, dtype=torch.uint8, device=self.device)
            self.v_scale = torch.empty(B * H * d, dtype=torch.float32, device=self.device)
        self.masks_built = False

    def build_masks(self, stream=None) -> None:
        for m in self.masks.values():
            m.build(self.geom, stream)
        self.masks_built = True

    def profile(self, q, k, v, sample_idx, stream=None) -> None:
        svg_profile_heads(self.geom, q, k, v, sample_idx, self.labels, self.mse, self.workspace,
                          n_samples=self.n_samples, stream=stream)

    def attend(self, q, k, v, o, lse=None, stream=None) -> None:
        """Permute temporal heads, block-sparse attention, un-permute (labels as set).

        lse, if given, is in frame-major rows on the fused layouts and in
        each head's own layout on the explicit one.
        """
        ms, mt = self.masks[SVG_MASK_SPATIAL], self.masks[SVG_MASK_TEMPORAL]
        if self.layout != "explicit":
            if self.layout == "fused":
                svg_permute_qkv(self.geom, None, k, v, None, self.kp, self.vp, self.labels,
                                stream=stream)
            svg_sparse_attention_fused(self.geom, q, k, v, self.kp, self.vp, self.labels,
                                       ms.row_ptr, ms.col_idx, mt.row_ptr, mt.col_idx, o, lse,
                                       stream=stream)
            return
        svg_permute_qkv(self.geom, q, k, v, self.qp, self.kp, self.vp, self.labels,
                        stream=stream)
        if self.pv == "e4m3":
            svg_quantize_v_e4m3(self.geom, v, self.vp, self.labels, self.v8, self.v_scale,
                                stream=stream)
            svg_sparse_attention_fp8pv(self.geom, q, k, self.qp, self.kp, self.v8, self.v_scale,
                                       self.labels, ms.row_ptr, ms.col_idx, mt.row_ptr,
                                       mt.col_idx, o, self.op, lse, stream=stream)
        else:
            svg_sparse_attention(self.geom, q, k, v, self.qp, self.kp, self.vp, self.labels,
                                 ms.row_ptr, ms.col_idx, mt.row_ptr, mt.col_idx, o, self.op, lse,
                                 stream=stream)
        svg_unpermute(self.geom, self.op, o, self.labels, stream=stream)

    def forward(self, q, k, v, sample_idx, o, lse=None, rebuild_masks: bool = False,
                stream=None) -> None:
        """The whole path: profile -> (masks) -> permute -> attention -> un-permute."""
        if rebuild_masks or not self.masks_built:
            self.build_masks(stream)
        self.profile(q, k, v, sample_idx, stream)
        self.attend(q, k, v, o, lse, stream)

    def dense(self, q, k, v, o, lse=None, stream=None) -> None:
        """The same attention kernel over the all-blocks mask (the dense baseline)."""
        if self.dense_mask is None:
            self.dense_mask = BlockMaskCSR(self.geom, SVG_MASK_DENSE, self.device)
            self.dense_mask.build(self.geom, stream)
        dm = self.dense_mask
        svg_sparse_attention(self.geom, q, k, v, None, None, None, None, dm.row_ptr, dm.col_idx,
                             None, None, o, None, lse, stream=stream)


class StreamedLayer:
    """The layer over a sequence of host-resident inputs, with copies overlapped.

    Each item is (q, k, v, sample_idx) in pinned host memory and an output
    buffer o in pinned host memory. Three CUDA streams form a pipeline over
    `depth` device buffer sets: while item i computes, the inputs of item i+1
    are copied in and the output of item i-1 is copied out. All compute of
    every item runs on one stream, so the layer's shared scratch (permuted
    tensors, labels, workspace, masks) is used by one item at a time.
    """

    def __init__(self, geom: Geom, n_samples: int, device="cuda", depth: int = 2):
        self.layer = SparseVideoGenLayer(geom, n_samples, device)
        dev = self.layer.device
        shape = (geom.B, geom.H, geom.N, geom.head_dim)
        self.depth = depth
        self.qkv = [tuple(torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(3))
                    for _ in range(depth)]
        self.rows = [torch.empty(n_samples, dtype=torch.int32, device=dev) for _ in range(depth)]
        self.out = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self.s_in = torch.cuda.Stream(dev)
        self.s_compute = torch.cuda.Stream(dev)
        self.s_out = torch.cuda.Stream(dev)
        mk = lambda: [torch.cuda.Event() for _ in range(depth)]  # noqa: E731
        self.ev_in, self.ev_done, self.ev_out = mk(), mk(), mk()
        self.started = [False] * depth
        with torch.cuda.stream(self.s_compute):
            self.layer.build_masks(stream=self.s_compute)

    def submit(self, i: int, q_h, k_h, v_h, rows_h, o_h) -> None:
        """Enqueues item number i (the caller numbers items 0, 1, 2, ...)."""
        b = i % self.depth
        q, k, v = self.qkv[b]
        if self.started[b]:
            self.s_in.wait_event(self.ev_done[b])  # inputs of the previous user computed
        with torch.cuda.stream(self.s_in):
            q.copy_(q_h, non_blocking=True)
            k.copy_(k_h, non_blocking=True)
            v.copy_(v_h, non_blocking=True)
            self.rows[b].copy_(rows_h, non_blocking=True)
            self.ev_in[b].record(self.s_in)
        self.s_compute.wait_event(self.ev_in[b])
        if self.started[b]:
            self.s_compute.wait_event(self.ev_out[b])  # output buffer copied out
        self.layer.forward(q, k, v, self.rows[b], self.out[b], stream=self.s_compute)
        self.ev_done[b].record(self.s_compute)
        self.s_out.wait_event(self.ev_done[b])
        with torch.cuda.stream(self.s_out):
            o_h.copy_(self.out[b], non_blocking=True)
            self.ev_out[b].record(self.s_out)
        self.started[b] = True

    def synchronize(self) -> None:
        for s in (self.s_in, self.s_compute, self.s_out):
            s.synchronize()


class SemanticSparseLayer:
    """Semantic-aware sparse attention (Sparse VideoGen 2) over one layer.

    The path (project article "Sparse-VideoGen and the sparsity hiding inside
    video diffusion attention", section "Three generations of the same idea"):
    k-means on the query and on the key vectors of every head, a stable
    cluster-sorted permutation of Q (by query cluster) and of K, V (by key
    cluster), the key clusters each query cluster keeps (top-p of the
    size-weighted centroid softmax), the tile pairs of the sorted layouts that
    hold a kept pair, block-sparse attention over them, and the output
    scattered back to the original order. This class owns the device buffers
    (allocated with torch) and calls the library in that order on one stream.
    """

    def __init__(self, B: int, H: int, N: int, d: int, Cq: int = 256, Ck: int = 256,
                 iters: int = 10, top_p: float = 0.9, block_k: int = 128, scale=None,
                 ear_tau: Optional[float] = None, device="cuda"):
        """ear_tau: None for Sparse VideoGen 2; a threshold for SVG-EAR (error-
        aware routing of skipped cluster pairs whose estimated error exceeds it,
        and centroid compensation of every key left out)."""
        from . import svg2_ear_workspace_bytes, svg2_kmeans_workspace_bytes
        self.B, self.H, self.N, self.d = B, H, N, d
        self.BH = B * H
        self.Cq, self.Ck, self.iters, self.top_p = Cq, Ck, iters, top_p
        self.block_q, self.block_k = 128, block_k
        self.scale = float(d ** -0.5 if scale is None else scale)
        dev = self.device = torch.device(device)
        BH = self.BH
        # the query and key clusterings run side by side on two streams, each
        # with its own workspace
        self.workspace = torch.empty(svg2_kmeans_workspace_bytes(BH, N, d, Cq) // 4 + 64,
                                     dtype=torch.float32, device=dev)
        self.workspace_k = torch.empty(svg2_kmeans_workspace_bytes(BH, N, d, Ck) // 4 + 64,
                                       dtype=torch.float32, device=dev)
        self._side = torch.cuda.Stream(device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.cq = torch.empty((BH, Cq, d), dtype=torch.float32, device=dev)
        self.ck = torch.empty((BH, Ck, d), dtype=torch.float32, device=dev)
        self.assign_q, self.assign_k = torch.empty((BH, N), **i32), torch.empty((BH, N), **i32)
        self.order_q, self.order_k = torch.empty((BH, N), **i32), torch.empty((BH, N), **i32)
        self.offsets_q = torch.empty((BH, Cq + 1), **i32)
        self.offsets_k = torch.empty((BH, Ck + 1), **i32)
        self.sel = torch.empty((BH, Cq, (Ck + 31) // 32), **i32)
        self.nqb = -(-N // self.block_q)
        self.nkb = -(-N // block_k)
        self.row_ptr = torch.empty(BH * self.nqb + 1, **i32)
        self.counts = torch.empty(BH * self.nqb, **i32)
        # every tile pair at most: the CSR never needs more
        self.col_idx = torch.empty(BH * self.nqb * self.nkb, **i32)
        shape = (self.B, self.H, N, d)
        self.qs, self.ks, self.vs, self.os = (torch.empty(shape, dtype=torch.bfloat16, device=dev)
                                              for _ in range(4))
        self.ear_tau = ear_tau
        if ear_tau is not None:
            self.vbar = torch.empty((BH, Ck, d), dtype=torch.float32, device=dev)
            self.disp = torch.empty((BH, Ck), dtype=torch.float32, device=dev)
            self.lse = torch.empty((BH, N), dtype=torch.float32, device=dev)
            self.ear_ws = torch.empty(svg2_ear_workspace_bytes(BH, d, Ck) // 4 + 64,
                                      dtype=torch.float32, device=dev)

    def plan(self, q, k, v=None, stream=None) -> None:
        """Clusters, permutations, selection and the tile CSR of q and k (and
        the value statistics of v for SVG-EAR's routing)."""
        if self.ear_tau is not None and v is None:
            raise ValueError("SVG-EAR routing needs v")
        self._v = v
        from . import svg2_build_tile_csr, svg2_kmeans, svg2_select_clusters
        BH, N, d = self.BH, self.N, self.d
        main = stream if stream is not None else torch.cuda.current_stream(self.device)
        if isinstance(main, int):
            main = torch.cuda.ExternalStream(main, device=self.device)
        # keys (and the value statistics) on the side stream, joined before the
        # selection; both start after what `main` holds so far (q, k, v written)
        side = self._side
        side.wait_stream(main)
        svg2_kmeans(BH, N, d, self.Cq, self.iters, q, self.cq, self.assign_q, self.order_q,
                    self.offsets_q, self.workspace, stream=main)
        svg2_kmeans(BH, N, d, self.Ck, self.iters, k, self.ck, self.assign_k, self.order_k,
                    self.offsets_k, self.workspace_k, stream=side)
        disp = None
        if self.ear_tau is not None:
            from . import svg2_cluster_value_stats
            svg2_cluster_value_stats(BH, N, d, self.Ck, self._v, self.order_k, self.offsets_k,
                                     self.vbar, self.disp, stream=side)
            disp = self.disp
        main.wait_stream(side)
        svg2_select_clusters(BH, d, self.Cq, self.Ck, self.scale, self.top_p, self.cq, self.ck,
                             self.offsets_k, self.sel, disp=disp, tau=self.ear_tau or 0.0,
                             stream=main)
        svg2_build_tile_csr(BH, N, self.Cq, self.Ck, self.block_q, self.block_k, self.offsets_q,
                            self.offsets_k, self.sel, self.row_ptr, self.col_idx, self.counts,
                            stream=main)

    def attend(self, q, k, v, o, lse=None, stream=None) -> None:
        """Permute, block-sparse attention over the planned tiles, un-permute."""
        from . import svg2_gather_rows, svg2_scatter_rows, svg2_sparse_attention
        BH, N, d = self.BH, self.N, self.d
        svg2_gather_rows(BH, N, d, q, self.order_q, self.qs, stream=stream)
        svg2_gather_rows(BH, N, d, k, self.order_k, self.ks, stream=stream)
        svg2_gather_rows(BH, N, d, v, self.order_k, self.vs, stream=stream)
        if self.ear_tau is None:
            svg2_sparse_attention(BH, N, d, self.block_k, self.scale, self.qs, self.ks, self.vs,
                                  self.row_ptr, self.col_idx, self.os, lse, stream=stream)
        else:
            from . import svg2_ear_compensate
            svg2_sparse_attention(BH, N, d, self.block_k, self.scale, self.qs, self.ks, self.vs,
                                  self.row_ptr, self.col_idx, self.os, self.lse, stream=stream)
            svg2_ear_compensate(BH, N, d, self.Ck, self.block_k, self.scale, self.qs, self.ck,
                                self.vbar, self.offsets_k, self.row_ptr, self.col_idx, self.os,
                                self.lse, self.ear_ws, stream=stream)
        svg2_scatter_rows(BH, N, d, self.os, self.order_q, o, stream=stream)

    def forward(self, q, k, v, o, lse=None, stream=None) -> None:
        self.plan(q, k, v, stream)
        self.attend(q, k, v, o, lse, stream)


def _on_stream(stream):
    """Context in which torch works on `stream`, of any kind that the calls take."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream))
    return torch.cuda.stream(stream)


class HistoryCache:
    """Keys and values of the frames made so far, and attention over them.

    A generator that makes a video chunk by chunk attends from each chunk to all
    frames before it. This class owns the page pools of `n_layers` layers, the
    page table they share and the workspaces (allocated with torch), and calls
    the library in order on one stream:

      reserve(seqs, counts)     room for a chunk's rows in every sequence of the batch
      write(layer, k, v)        a layer's keys and values of the chunk (again at
                                each denoising step: the rows are overwritten),
                                until the next fork, free, reset or compact
      attend(layer, q, ...)     the chunk's queries over the shared history and
                                each sequence's own rows
      fork(src, dst)            continuations of one history, sharing its pages
      free(seqs, keep)          a sequence dropped, or cut back to its first rows
      compact()                 the pages in use moved to the front of the pools
      check()                   an error if any of these was refused on the device

    What depends on the state is refused on the device, with no word from the call itself: a reserve
    without enough free pages reserves nothing, after which write writes nothing and attend
    reads the lengths as they were. check() tells, at the price of a wait: call it after
    reserve where the pools may run out, or once a chunk.

    seqs, counts, src, dst and keep are device int32 tensors; negative sequence
    numbers are idle entries of a padded batch. One cache is used by one stream
    at a time, by one captured graph at a time as well.
    """

    def __init__(self, n_layers: int, n_pages: int, page_size: int, H: int, H_kv: int, d: int,
                 max_seqs: int, max_rows: int, batch: int, rows: int, scale=None, device="cuda"):
        """max_rows: of one sequence, at most 2^20; batch, rows: the most sequences and query
        rows a sequence that one call of reserve, write or attend has. device: the current one,
        here and in every call, as everywhere in this library; the pools are set up on its
        current stream."""
        from . import CacheGeom, svg_cache_reset, svg_prefix_attention_workspace_bytes
        dev = self.device = torch.device(device)
        if dev.type == "cuda" and dev.index is not None and dev.index != torch.cuda.current_device():
            raise ValueError(f"the current device is cuda:{torch.cuda.current_device()}: make {dev} the "
                             f"current one (torch.cuda.device) for a cache there")
        self.geom = CacheGeom(n_pages, page_size, H_kv, d, max_seqs, -(-max_rows // page_size))
        self.H = H
        self.scale = float(d ** -0.5 if scale is None else scale)
        need = svg_prefix_attention_workspace_bytes(self.geom, batch, H, rows)
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.empty((max_seqs, self.geom.max_pages), **i32)
        self.lens, self.refs = torch.empty(max_seqs, **i32), torch.empty(n_pages, **i32)
        self.plan = torch.empty((batch, 4), **i32)
        self._numbers = torch.empty(batch, **i32)  # of the sequences the plan is for
        self.moves = torch.empty(2 + 2 * n_pages, **i32)
        shape = (n_pages, H_kv, page_size, d)
        mk = lambda: torch.empty(shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.pools = [(mk(), mk()) for _ in range(n_layers)]
        self._planned = 0  # entries of the plan; 0: none, or one of an earlier state
        svg_cache_reset(self.geom, self.table, self.lens, self.refs)

    @property
    def _state(self):
        return self.table, self.lens, self.refs

    def reset(self, stream=None) -> None:
        from . import svg_cache_reset
        svg_cache_reset(self.geom, *self._state, stream=stream)
        self._planned = 0  # the plan is of the state before

    def fork(self, src, dst, stream=None) -> None:
        from . import svg_cache_fork
        svg_cache_fork(self.geom, *self._state, src, dst, stream=stream)
        self._planned = 0  # a target may share the rows of the plan

    def free(self, seqs, keep=None, stream=None) -> None:
        from . import svg_cache_free
        svg_cache_free(self.geom, *self._state, seqs, keep, stream=stream)
        self._planned = 0  # the plan's rows may be gone

    def reserve(self, seqs, counts, stream=None) -> None:
        """All of it or, where the pools have too few free pages, nothing (see check)."""
        from . import svg_cache_reserve
        svg_cache_reserve(self.geom, *self._state, seqs, counts, self.plan, stream=stream)
        # write pairs the plan with these numbers, whatever the caller's list holds by then
        n = seqs.numel()
        numbers = self._numbers if n == self._numbers.numel() else self._numbers[:n]
        if stream is None:
            numbers.copy_(seqs.view(n))
        else:
            with _on_stream(stream):
                numbers.copy_(seqs.view(n))
        self._planned = n

    def check(self, stream=None) -> None:
        """Waits for the stream and raises SvgError if something was refused on the current
        device since the status was last read (by this or by svg_get_device_status):
        SVG_ERR_CAPACITY where reserve had no room, SVG_ERR_INVALID_ARG for a sequence
        number or a state that cannot be, SVG_ERR_DEVICE_TIMEOUT. Not while a graph is captured."""
        from . import SVG_OK, SvgError, svg_get_device_status
        status, _ = svg_get_device_status(stream)
        if status != SVG_OK:
            raise SvgError("HistoryCache", status)

    def write(self, layer: int, k_new, v_new, stream=None) -> None:
        """k_new, v_new [n, H_kv, L, d]: the rows that the last reserve made room for."""
        from . import svg_cache_write
        if not self._planned:
            raise ValueError("write follows reserve, with no fork, free, reset or compact between")
        n, H_kv, _, d = k_new.shape
        if v_new.shape != k_new.shape or H_kv != self.geom.H_kv or d != self.geom.head_dim \
                or n != self._planned:
            raise ValueError(f"rows of shape {tuple(k_new.shape)} and {tuple(v_new.shape)} for "
                             f"{self._planned} sequences, {self.geom.H_kv} heads of "
                             f"{self.geom.head_dim}")
        svg_cache_write(self.geom, self.table, self._numbers, self.plan, k_new.shape[2], k_new, v_new,
                        *self.pools[layer], n=n, stream=stream)

    def compact(self, stream=None) -> None:
        from . import svg_cache_compact, svg_cache_copy_pages
        svg_cache_compact(self.geom, self.table, self.refs, self.table, self.refs, self.moves,
                          stream=stream)
        for k, v in self.pools:
            svg_cache_copy_pages(self.geom, self.moves, self.geom.n_pages, k, v, k, v,
                                 stream=stream)
        self._planned = 0  # the plan names pages by their old numbers

    def attend(self, layer: int, q, seqs, prefix_seq: int, prefix_len: int, o, lse=None,
               stream=None) -> None:
        """q, o [B, H, Lq, d]; the first prefix_len rows of prefix_seq are shared by all."""
        from . import svg_prefix_attention
        B, H, Lq, d = q.shape
        if o.shape != q.shape or H != self.H or d != self.geom.head_dim or B != seqs.numel() \
                or (lse is not None and lse.shape != q.shape[:3]):
            raise ValueError(f"queries of shape {tuple(q.shape)}, outputs of shape {tuple(o.shape)} "
                             f"for {seqs.numel()} sequences, {self.H} heads of {self.geom.head_dim}")
        svg_prefix_attention(self.geom, q.shape[0], self.H, q.shape[2], prefix_seq, prefix_len,
                             self.scale, q, *self.pools[layer], self.table, self.lens, seqs, o,
                             lse, self.workspace, stream=stream)
