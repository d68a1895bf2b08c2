// Attention of a batch of sequences over the history they share and each
// one's own rows after it, keys and values read from cache pages.
//
// O_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i), s = scale q.k, with
// the maximum m and both sums carried over the keys in one pass.
//
// First form: one warp per query row, a key at a time. Every row reads every
// key, so it is bound by L2 traffic and by the reduction over the lanes.
#include "internal.h"
#include "sm100.cuh"

namespace svg {
namespace {

constexpr int kRowWarps = 4;

struct RowParams {
  CacheDims c;
  int32_t B, H, Lq, prefix_seq, prefix_len;
  float scale_log2;
  const svg_bf16 *q, *k_pages, *v_pages;
  const int32_t *table, *lens, *seqs;
  svg_bf16* o;
  float* lse;
  int* status;
};

__device__ __forceinline__ float bf16_to_float(svg_bf16 x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) prefix_row_kernel(const RowParams p) {
  constexpr int kE = D / 32;
  const int lane = lane_id();
  const int64_t row = blockIdx.x * static_cast<int64_t>(kRowWarps) + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.H * p.Lq) return;
  const int64_t bh = row / p.Lq;
  const int b = static_cast<int>(bh / p.H), kv = static_cast<int>(bh % p.H) / (p.H / p.c.H_kv);
  const int seq = p.seqs[b];
  if (seq < 0) return;  // idle entry: its rows stay as they are
  int len = 0;
  if (seq < p.c.max_seqs) len = p.lens[seq];
  if (seq >= p.c.max_seqs || len < 0 || len > p.c.max_rows()) {
    if (lane == 0) atomicOr(p.status, kDevErrBounds);
    return;
  }
  if (p.prefix_len > 0) {
    const int have = p.lens[p.prefix_seq];
    if (have < p.prefix_len || have > p.c.max_rows()) {
      if (lane == 0) atomicOr(p.status, kDevErrBounds);
      return;
    }
  }
  float q[kE], o[kE], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = bf16_to_float(p.q[row * D + e * 32 + lane]) * p.scale_log2;
    o[e] = 0.0f;
  }
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? 0 : p.prefix_len, hi = part == 0 ? p.prefix_len : len;
    const int32_t* pages = p.table + static_cast<int64_t>(part == 0 ? p.prefix_seq : seq) * p.c.max_pages;
    for (int j = lo; j < hi; ++j) {
      const int page = pages[j / p.c.ps];
      const bool bad = page < 0 || page >= p.c.n_pages;
      if (bad && lane == 0) atomicOr(p.status, kDevErrBounds);
      const int64_t at =
          bad ? 0 : ((static_cast<int64_t>(page) * p.c.H_kv + kv) * p.c.ps + j % p.c.ps) * D;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < kE; ++e) s += q[e] * (bad ? 0.0f : bf16_to_float(p.k_pages[at + e * 32 + lane]));
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      const float m_new = fmaxf(m, s);
      const float alpha = fast_exp2(m - m_new), w = fast_exp2(s - m_new);
      l = l * alpha + w;
      m = m_new;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        o[e] = o[e] * alpha + w * (bad ? 0.0f : bf16_to_float(p.v_pages[at + e * 32 + lane]));
    }
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float x = l > 0.0f ? o[e] / l : 0.0f;
    p.o[row * D + e * 32 + lane] = static_cast<svg_bf16>(pack_bf16x2(x, 0.0f) & 0xffffu);
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = l > 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t prefix_workspace_bytes(const CacheDims&, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_prefix_attention(const PrefixArgs& a, int* status, cudaStream_t stream) {
  RowParams p{a.c,     a.B,       a.H,       a.Lq,    a.prefix_seq, a.prefix_len,
              a.scale * 1.4426950408889634f, a.q,     a.k_pages,    a.v_pages,
              a.table, a.lens,    a.seqs,    a.o,     a.lse,        status};
  const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.Lq;
  const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
  auto kern = a.c.d == 128 ? prefix_row_kernel<128> : prefix_row_kernel<64>;
  kern<<<grid, kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace svg
