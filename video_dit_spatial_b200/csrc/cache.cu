// The pages of a history cache: keys and values of rows (frames) made earlier,
// kept in pages that several sequences share.
//
// State, all in caller memory: a page table [max_seqs, max_pages], a length per
// sequence, and a reference count per page. A page is free when its count is
// zero; there is no free list, so nothing has to be kept in order: pages are
// handed out lowest number first, which makes every call's result depend on
// the state and its arguments alone. The bookkeeping kernels touch integers
// only and are bound by the latency of a few dependent loads (2 to 5 us, with many
// sequences of many shared pages by the atomics on their counts); the two
// kernels that move rows are bound by HBM: 709 MB written in 103 us (6.9 TB/s, the last of
// it into L2), 1.57 GB of pages copied in 242 us (6.5 TB/s).
#include "internal.h"
#include "sm100.cuh"

namespace svg {
namespace {

constexpr int kRowThreads = 256;
// fork and free: a CTA per sequence, a page per thread in one step for most
// sequences (the atomics' latency is what a step costs: 64 sequences of 929
// pages took 13.5 us at 256 threads).
constexpr int kSeqThreads = 1024;

__device__ __forceinline__ void flag(int* status, int bit) { atomicOr(status, bit); }

__global__ void cache_reset_kernel(CacheDims c, int32_t* table, int32_t* lens, int32_t* refs) {
  const int64_t n = static_cast<int64_t>(c.max_seqs) * c.max_pages;
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = i0; i < n; i += step) table[i] = -1;
  for (int64_t i = i0; i < c.max_seqs; i += step) lens[i] = 0;
  for (int64_t i = i0; i < c.n_pages; i += step) refs[i] = 0;
}

// One CTA per entry. Every CTA finds by itself whether its entry is to be
// refused (an earlier entry has the same target, or its source is a target of
// the call), so no CTA reads what another one writes.
__global__ void __launch_bounds__(kSeqThreads)
    cache_fork_kernel(CacheDims c, int32_t* table, int32_t* lens, int32_t* refs,
                      const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                      int* status) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int s = src[i], t = dst[i];
  if (s < 0 || t < 0) return;  // idle entry
  bool bad = s >= c.max_seqs || t >= c.max_seqs;
  for (int j = tid; j < n; j += kSeqThreads) {
    const int tj = src[j] < 0 ? -1 : dst[j];
    bad = bad || (j < i && tj == t) || tj == s;
  }
  bad = __syncthreads_or(bad);
  int len = 0;
  if (!bad) {
    len = lens[s];
    bad = len < 0 || len > c.max_rows() || lens[t] != 0;
  }
  if (bad) {
    if (tid == 0) flag(status, kDevErrBounds);
    return;
  }
  const int used = (len + c.ps - 1) / c.ps;
  const int32_t* from = table + static_cast<int64_t>(s) * c.max_pages;
  int32_t* to = table + static_cast<int64_t>(t) * c.max_pages;
  // A page number that cannot be refuses the entry: all are looked at before the first is copied.
  const int p0 = tid < used ? from[tid] : 0;
  for (int k = tid; k < used; k += kSeqThreads) {
    const int p = k == tid ? p0 : from[k];
    bad = bad || p < 0 || p >= c.n_pages;
  }
  if (__syncthreads_or(bad)) {  // every thread has read lens[t], too
    if (tid == 0) flag(status, kDevErrBounds);
    return;
  }
  for (int k = tid; k < used; k += kSeqThreads) {
    const int p = k == tid ? p0 : from[k];
    to[k] = p;
    atomicAdd(refs + p, 1);
  }
  if (tid == 0) lens[t] = len;
}

__global__ void __launch_bounds__(kSeqThreads)
    cache_free_kernel(CacheDims c, int32_t* table, int32_t* lens, int32_t* refs,
                      const int32_t* __restrict__ seqs, const int32_t* __restrict__ keep, int n,
                      int* status) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int s = seqs[i];
  if (s < 0) return;  // idle entry
  const int kept = keep != nullptr ? keep[i] : 0;
  bool bad = s >= c.max_seqs || kept < 0;
  for (int j = tid; j < i; j += kSeqThreads) bad = bad || seqs[j] == s;
  bad = __syncthreads_or(bad);
  int len = 0;
  if (!bad) {
    len = lens[s];
    bad = len < 0 || len > c.max_rows();
  }
  if (bad) {
    if (tid == 0) flag(status, kDevErrBounds);
    return;
  }
  if (kept >= len) return;
  int32_t* mine = table + static_cast<int64_t>(s) * c.max_pages;
  const int used = (len + c.ps - 1) / c.ps;
  for (int k = (kept + c.ps - 1) / c.ps + tid; k < used; k += kSeqThreads) {
    const int p = mine[k];
    mine[k] = -1;
    if (p < 0 || p >= c.n_pages) {
      flag(status, kDevErrBounds);
    } else if (atomicSub(refs + p, 1) <= 0) {  // not in use: leave it free
      atomicAdd(refs + p, 1);
      flag(status, kDevErrBounds);
    }
  }
  __syncthreads();  // every thread has read lens[s]
  if (tid == 0) lens[s] = kept;
}

// ---------------------------------------------------------------- one-CTA bookkeeping
constexpr int kOneThreads = 1024;
constexpr int kPer = 16;                      // pages a thread looks at per step
constexpr int kStep = kOneThreads * kPer;     // pages the CTA looks at per step

// Inclusive sum over the CTA's threads; `total` gets the whole sum.
__device__ __forceinline__ int block_sum_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums free again
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return x + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Bit k: page p0 + k of the pool is in use; pages past the end count as in use
// or free as `past` says.
__device__ __forceinline__ uint32_t used_bits(const int32_t* refs, int p0, int n_pages, bool past) {
  uint32_t m = 0;
  if (p0 + kPer <= n_pages) {  // refs is 16-byte aligned, p0 a multiple of 16
    int4 r[kPer / 4];
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) r[q] = reinterpret_cast<const int4*>(refs + p0)[q];
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q)
      m |= ((r[q].x > 0 ? 1u : 0u) | (r[q].y > 0 ? 2u : 0u) | (r[q].z > 0 ? 4u : 0u) |
            (r[q].w > 0 ? 8u : 0u))
           << (4 * q);
  } else {
    for (int k = 0; k < kPer; ++k) {
      const bool used = p0 + k < n_pages ? refs[p0 + k] > 0 : past;
      m |= used ? 1u << k : 0u;
    }
  }
  return m;
}

// One CTA: thread i holds entry i. The wanted pages are counted and summed
// over the entries, the free pages counted (as far as needed), and only when
// they suffice is anything written.
__global__ void __launch_bounds__(kOneThreads)
    cache_reserve_kernel(CacheDims c, int32_t* table, int32_t* lens, int32_t* refs,
                         const int32_t* __restrict__ seqs, const int32_t* __restrict__ counts,
                         int n, int32_t* plan, int* status) {
  __shared__ int s_seq[kOneThreads], s_off[kOneThreads], s_slot[kOneThreads];
  __shared__ uint16_t s_free[kStep];  // the step's free pages, ascending, relative to its first
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  int s = -1, add = 0, len = 0, open = -1, slot = 0, need = 0;
  bool cow = false;
  // The counts of the first step's pages, loaded beside the entries; most pools have no more.
  const uint32_t first_free =
      tid * kPer < c.n_pages ? ~used_bits(refs, tid * kPer, c.n_pages, true) & ((1u << kPer) - 1u)
                             : 0u;
  if (tid < n) {
    s = seqs[tid];
    add = counts[tid];
  }
  if (s < 0) add = 0;  // idle entry
  s_seq[tid] = s;
  __syncthreads();
  if (s >= 0) {
    bool bad = s >= c.max_seqs || add < 0;
    for (int j = 0; j < tid && !bad; ++j) bad = s_seq[j] == s;
    if (!bad) {
      len = lens[s];
      bad = len < 0 || len > c.max_rows();
    }
    if (!bad && add > c.max_rows() - len) {
      flag(status, kDevErrCapacity);
      add = 0;
    }
    if (!bad && add > 0) {
      slot = (len + c.ps - 1) / c.ps;
      need = (len + add + c.ps - 1) / c.ps - slot;
      if (len % c.ps != 0) {
        open = table[static_cast<int64_t>(s) * c.max_pages + len / c.ps];
        if (open < 0 || open >= c.n_pages) {
          bad = true;
        } else if (refs[open] > 1) {  // others read this page: a copy of it is written instead
          cow = true;
          slot -= 1;
          need += 1;
        }
      }
    }
    if (bad) {
      flag(status, kDevErrBounds);
      add = need = 0;
      cow = false;
    }
  }
  // An entry wants max_pages pages at most and no sequence has two entries that want any: the sum
  // is at most max_seqs * max_pages, which fits 32 bits.
  int total;
  s_off[tid] = block_sum_scan(need, warp_sums, total) - need;
  s_slot[tid] = slot;
  // pass 0 counts the free pages, pass 1 hands them out
  bool enough = total == 0;
  for (int pass = 0; pass < 2 && total > 0; ++pass) {
    int base = 0;
    for (int p0 = 0; p0 < c.n_pages && base < total; p0 += kStep) {
      const int mine = p0 + tid * kPer;
      uint32_t free_bits = first_free;
      if (p0 > 0)
        free_bits =
            mine < c.n_pages ? ~used_bits(refs, mine, c.n_pages, true) & ((1u << kPer) - 1u) : 0u;
      int found;
      int at = block_sum_scan(__popc(free_bits), warp_sums, found) - __popc(free_bits);
      if (pass == 1) {
        for (; free_bits != 0; free_bits &= free_bits - 1)
          s_free[at++] = static_cast<uint16_t>(tid * kPer + __ffs(free_bits) - 1);
        __syncthreads();
        // the refs this step reads are written only now, and no later step reads them
        for (int k = tid; k < found && base + k < total; k += kOneThreads) {
          const int r = base + k, page = p0 + s_free[k];
          int lo = 0, hi = n - 1;  // the last entry whose pages start at or before rank r
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_off[mid] <= r) {
              lo = mid;
            } else {
              hi = mid - 1;
            }
          }
          table[static_cast<int64_t>(s_seq[lo]) * c.max_pages + s_slot[lo] + r - s_off[lo]] = page;
          refs[page] = 1;
        }
        __syncthreads();  // s_free is filled again by the next step
      }
      base += found;
    }
    if (pass == 0) {
      enough = base >= total;
      if (!enough) break;
    }
  }
  __syncthreads();  // the table entries written above are read below
  if (tid < n) {
    int32_t* out = plan + 4 * static_cast<int64_t>(tid);
    if (!enough) add = 0;
    out[0] = len;
    out[1] = add;
    out[2] = enough && cow ? open : -1;
    out[3] = enough && cow ? table[static_cast<int64_t>(s) * c.max_pages + slot] : -1;
    if (enough && cow) atomicSub(refs + open, 1);
    if (add > 0) lens[s] = len + add;
  }
  if (!enough && tid == 0) flag(status, kDevErrCapacity);
}

// One CTA: the number of pages in use, the free pages below that number and
// the pages in use from it on, both ascending and equally many: the i-th of
// one takes the i-th of the other.
__global__ void __launch_bounds__(kOneThreads)
    cache_compact_kernel(CacheDims c, const int32_t* __restrict__ refs, int32_t* moves) {
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  int live = 0;
  for (int p0 = 0; p0 < c.n_pages; p0 += kStep) {
    const int mine = p0 + tid * kPer;
    const uint32_t used = mine < c.n_pages ? used_bits(refs, mine, c.n_pages, false) : 0u;
    int found;
    block_sum_scan(__popc(used), warp_sums, found);
    live += found;
  }
  int32_t* to = moves + 2 + c.n_pages;  // where each page goes; -1: it is free
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < c.n_pages; p0 += kStep) {
    const int mine = p0 + tid * kPer;
    const uint32_t used = mine < c.n_pages ? used_bits(refs, mine, c.n_pages, false) : 0u;
    // bits of this thread's pages below `live`
    const int below = min(max(live - mine, 0), kPer);
    const uint32_t low = (1u << below) - 1u;
    uint32_t hole = ~used & low, mover = used & ~low;
    int found;
    int at = holes + block_sum_scan(__popc(hole), warp_sums, found) - __popc(hole);
    for (; hole != 0; hole &= hole - 1) moves[3 + 2 * at++] = mine + __ffs(hole) - 1;
    holes += found;
    at = movers + block_sum_scan(__popc(mover), warp_sums, found) - __popc(mover);
    for (; mover != 0; mover &= mover - 1) moves[2 + 2 * at++] = mine + __ffs(mover) - 1;
    movers += found;
    for (int k = 0; k < kPer && mine + k < c.n_pages; ++k)
      to[mine + k] = k < below && (used >> k & 1u) ? mine + k : -1;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += kOneThreads) to[moves[2 + 2 * i]] = moves[3 + 2 * i];
  if (tid == 0) {
    moves[0] = movers;
    moves[1] = live;
  }
}

// The table and the counts after the moves. Each page's count is written by
// one thread, and a moved page's is read by the thread that clears it, so the
// outputs may be the inputs.
__global__ void cache_renumber_kernel(CacheDims c, const int32_t* table, const int32_t* refs,
                                      int32_t* table_out, int32_t* refs_out,
                                      const int32_t* __restrict__ moves, int* status) {
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int n_moves = moves[0], live = moves[1];
  const int32_t* to = moves + 2 + c.n_pages;
  const int64_t n = static_cast<int64_t>(c.max_seqs) * c.max_pages;
  for (int64_t i = i0; i < n; i += step) {
    const int p = table[i];
    const int q = p < 0 ? p : p < c.n_pages ? to[p] : -1;
    if (q < 0 && p >= 0) flag(status, kDevErrBounds);  // not a page in use
    table_out[i] = q;
  }
  for (int64_t i = i0; i < n_moves; i += step) {
    const int from = moves[2 + 2 * i], at = moves[3 + 2 * i];
    refs_out[at] = refs[from];
    refs_out[from] = 0;
  }
  for (int64_t i = i0; i < c.n_pages; i += step) {
    const int r = refs[i];
    if (i < live ? r > 0 : r <= 0) refs_out[i] = r;
  }
}

// ---------------------------------------------------------------- rows and pages
// A CTA moves 16 KB of keys and 16 KB of values, each thread eight 16-byte
// vectors that it loads before it stores the first.
constexpr int kPasses = 4;
constexpr int kChunkVecs = kRowThreads * kPasses;  // 16-byte vectors of one tensor

// grid: (row chunks of the new rows, then of a page; kv heads; entries). A
// chunk of the second kind copies the rows of a replaced open page.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
    cache_write_kernel(CacheDims c, const int32_t* __restrict__ table,
                       const int32_t* __restrict__ seqs, const int32_t* __restrict__ plan, int L,
                       int new_chunks, const uint4* __restrict__ k_new,
                       const uint4* __restrict__ v_new, uint4* k_pages, uint4* v_pages,
                       int* status) {
  constexpr int kVecs = D / 8;  // vectors of a row
  constexpr int kRowsPerPass = kRowThreads / kVecs;
  const int i = blockIdx.z, h = blockIdx.y;
  const int s = seqs[i];
  if (s < 0) return;
  const int first = plan[4 * i], count = plan[4 * i + 1];
  const int cow_src = plan[4 * i + 2], cow_dst = plan[4 * i + 3];
  const bool copy = static_cast<int>(blockIdx.x) >= new_chunks;
  const int chunk = copy ? blockIdx.x - new_chunks : blockIdx.x;
  bool bad = s >= c.max_seqs || first < 0 || count < 0 || count > L || first > c.max_rows() - count;
  const bool none = cow_src < 0 && cow_dst < 0;
  bad = bad || (!none && (cow_src < 0 || cow_dst < 0 || cow_src >= c.n_pages || cow_dst >= c.n_pages));
  if (bad) {  // every chunk of the entry finds the same
    if (threadIdx.x == 0) flag(status, kDevErrBounds);
    return;
  }
  if (copy && none) return;
  const int vec = threadIdx.x % kVecs;
  const int row0 = chunk * kRowsPerPass * kPasses + threadIdx.x / kVecs;
  const int rows = copy ? first % c.ps : count;
  const uint4* ks = copy ? k_pages : k_new;
  const uint4* vs = copy ? v_pages : v_new;
  const int64_t from0 = copy ? (static_cast<int64_t>(cow_src) * c.H_kv + h) * c.ps
                             : (static_cast<int64_t>(i) * c.H_kv + h) * L;
  uint4 kx[kPasses], vx[kPasses];
  int64_t to[kPasses];
#pragma unroll
  for (int q = 0; q < kPasses; ++q) {
    const int row = row0 + q * kRowsPerPass;
    to[q] = -1;
    if (row >= rows) continue;
    int page = cow_dst, at = row;
    if (!copy) {
      at = (first + row) % c.ps;
      page = table[static_cast<int64_t>(s) * c.max_pages + (first + row) / c.ps];
      if (page < 0 || page >= c.n_pages) {
        flag(status, kDevErrBounds);
        continue;
      }
    }
    const int64_t from = (from0 + row) * kVecs + vec;
    kx[q] = ks[from];
    vx[q] = vs[from];
    to[q] = ((static_cast<int64_t>(page) * c.H_kv + h) * c.ps + at) * kVecs + vec;
  }
#pragma unroll
  for (int q = 0; q < kPasses; ++q) {
    if (to[q] < 0) continue;
    k_pages[to[q]] = kx[q];
    v_pages[to[q]] = vx[q];
  }
}

// Whole pages, as listed (moves[2 + 2i] -> moves[3 + 2i]); a page is one run of
// memory, cut into chunks over a grid of fixed size, since the number of moves
// is only known on the device.
__global__ void __launch_bounds__(kRowThreads)
    cache_copy_kernel(CacheDims c, const int32_t* __restrict__ moves, int max_moves,
                      const uint4* k_src, const uint4* v_src, uint4* k_dst, uint4* v_dst,
                      int* status) {
  int n = moves[0];
  if (n < 0 || n > max_moves) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag(status, kDevErrBounds);
    n = n < 0 ? 0 : max_moves;
  }
  const int64_t page_vecs = static_cast<int64_t>(c.H_kv) * c.ps * (c.d / 8);
  const int64_t chunks = (page_vecs + kChunkVecs - 1) / kChunkVecs;
  for (int64_t w = blockIdx.x; w < n * chunks; w += gridDim.x) {
    const int i = static_cast<int>(w / chunks);
    const int from = moves[2 + 2 * i], to = moves[3 + 2 * i];
    if (from < 0 || to < 0 || from >= c.n_pages || to >= c.n_pages) {
      if (threadIdx.x == 0) flag(status, kDevErrBounds);
      continue;
    }
    const int64_t v0 = (w % chunks) * kChunkVecs + threadIdx.x;
    uint4 kx[kPasses], vx[kPasses];
#pragma unroll
    for (int q = 0; q < kPasses; ++q)
      if (v0 + q * kRowThreads < page_vecs) {
        kx[q] = k_src[from * page_vecs + v0 + q * kRowThreads];
        vx[q] = v_src[from * page_vecs + v0 + q * kRowThreads];
      }
#pragma unroll
    for (int q = 0; q < kPasses; ++q)
      if (v0 + q * kRowThreads < page_vecs) {
        k_dst[to * page_vecs + v0 + q * kRowThreads] = kx[q];
        v_dst[to * page_vecs + v0 + q * kRowThreads] = vx[q];
      }
  }
}

inline unsigned grid_for(int64_t n, int64_t per, int64_t most) {
  const int64_t g = (n + per - 1) / per;
  return static_cast<unsigned>(g < 1 ? 1 : (g < most ? g : most));
}

}  // namespace

cudaError_t launch_cache_reset(const CacheDims& c, int32_t* table, int32_t* lens, int32_t* refs,
                               cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(c.max_seqs) * c.max_pages + c.n_pages;
  cache_reset_kernel<<<grid_for(n, 1024, 1184), 256, 0, stream>>>(c, table, lens, refs);
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheDims& c, int32_t* table, int32_t* lens, int32_t* refs,
                              const int32_t* src, const int32_t* dst, int32_t n, int* status,
                              cudaStream_t stream) {
  cache_fork_kernel<<<n, kSeqThreads, 0, stream>>>(c, table, lens, refs, src, dst, n, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheDims& c, int32_t* table, int32_t* lens, int32_t* refs,
                              const int32_t* seqs, const int32_t* keep, int32_t n, int* status,
                              cudaStream_t stream) {
  cache_free_kernel<<<n, kSeqThreads, 0, stream>>>(c, table, lens, refs, seqs, keep, n, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_reserve(const CacheDims& c, int32_t* table, int32_t* lens, int32_t* refs,
                                 const int32_t* seqs, const int32_t* counts, int32_t n,
                                 int32_t* plan, int* status, cudaStream_t stream) {
  cache_reserve_kernel<<<1, kOneThreads, 0, stream>>>(c, table, lens, refs, seqs, counts, n, plan,
                                                      status);
  return cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheDims& c, const int32_t* table, const int32_t* seqs,
                               const int32_t* plan, int32_t n, int32_t L, const svg_bf16* k_new,
                               const svg_bf16* v_new, svg_bf16* k_pages, svg_bf16* v_pages,
                               int* status, cudaStream_t stream) {
  const int rows = kChunkVecs / (c.d / 8);  // rows of a chunk
  const int new_chunks = (L + rows - 1) / rows;
  const dim3 grid(new_chunks + (c.ps + rows - 1) / rows, c.H_kv, n);
  auto kern = c.d == 128 ? cache_write_kernel<128> : cache_write_kernel<64>;
  kern<<<grid, kRowThreads, 0, stream>>>(
      c, table, seqs, plan, L, new_chunks, reinterpret_cast<const uint4*>(k_new),
      reinterpret_cast<const uint4*>(v_new), reinterpret_cast<uint4*>(k_pages),
      reinterpret_cast<uint4*>(v_pages), status);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheDims& c, const int32_t* table, const int32_t* refs,
                                 int32_t* table_out, int32_t* refs_out, int32_t* moves, int* status,
                                 cudaStream_t stream) {
  cache_compact_kernel<<<1, kOneThreads, 0, stream>>>(c, refs, moves);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(c.max_seqs) * c.max_pages + c.n_pages;
  cache_renumber_kernel<<<grid_for(n, 1024, 1184), 256, 0, stream>>>(c, table, refs, table_out,
                                                                     refs_out, moves, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(const CacheDims& c, const int32_t* moves, int32_t max_moves,
                              const svg_bf16* k_src, const svg_bf16* v_src, svg_bf16* k_dst,
                              svg_bf16* v_dst, int* status, cudaStream_t stream) {
  const int64_t page_vecs = static_cast<int64_t>(c.H_kv) * c.ps * (c.d / 8);
  const int64_t chunks = (page_vecs + kChunkVecs - 1) / kChunkVecs * max_moves;
  cache_copy_kernel<<<grid_for(chunks, 1, 148 * 8), kRowThreads, 0, stream>>>(
      c, moves, max_moves, reinterpret_cast<const uint4*>(k_src),
      reinterpret_cast<const uint4*>(v_src), reinterpret_cast<uint4*>(k_dst),
      reinterpret_cast<uint4*>(v_dst), status);
  return cudaGetLastError();
}

}  // namespace svg
