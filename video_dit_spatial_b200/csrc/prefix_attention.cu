// Attention of a batch of sequences over the history they share and each
// one's own rows after it, keys and values read from cache pages.
//
// O_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i), s = scale q.k: one
// pass over the keys with a running maximum and sum per row. Two disjoint key
// sets give (O, m, l) each, joined exactly by
//   m = max(m1, m2), l = sum l_k 2^(m_k - m), O = sum O_k 2^(m_k - m) / l,
// which is what makes the work divisible along the keys.
//
// Work. With G = H / H_kv query heads to a key head, the G * Lq query rows of
// (sequence b, key head) are contiguous in q. Items, each a group of up to 256
// rows and a list of 128-key blocks:
//   shared    (key head, group of the rows of ALL sequences) x the prefix;
//   own       (key head, sequence, group of its rows) x its own rows after the
//             prefix, or, when the rows of one sequence fill the groups by
//             themselves (joint), x the prefix and then its own rows.
// The blocks of all items, in order, are one line of cost, cut into one
// equal piece per CTA: every SM gets the same work whatever the lengths
// are, which only the device knows. A piece begins and ends anywhere in an
// item; what a CTA has of an item that is not whole is written as (O, m, l) in
// fp32 and joined by a second kernel.
//
// One CTA per SM walks its piece. 384 threads: warps 0-3 and 4-7 softmax
// and epilogue (thread = row = tensor-memory lane), warp 8 TMA producer, warp 9
// MMA issuer, warps 10-11 load query rows. Two forms of an item:
//   two tiles  129..256 rows: tile A and tile B, each block serves both;
//   one tile   up to 128 rows: tile A and tile B hold the SAME rows, A takes
//              the even blocks and B the odd ones, so that one's softmax
//              overlaps the other's products, and the two are joined in the epilogue.
// Tensor memory: S_A 0, O_A 128, S_B 256, O_B 384; P (bf16) overwrites S. The
// weights are rounded to bf16 because the tensor core multiplies them with bf16 values
// (off by at most 2^-8 of each); row sums are taken before that rounding, in
// fp32, as are the maxima and O.
#include <cstring>

#include "internal.h"
#include "sm100.cuh"

namespace svg {
namespace {

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kLoadThreads = 64;  // warps 10 and 11
constexpr int kLaunchRegs = 168;
constexpr int kSoftmaxRegs = 224;
constexpr int kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * kLaunchRegs, "register split");
constexpr float kRebaseLog2 = 8.0f;  // O is re-based when a maximum grows by more than 2^8
constexpr int kBK = 128;             // keys of a block
constexpr int kGroup = 256;          // rows of an item
constexpr int kMaxCtas = 148;
constexpr int kMaxBatch = 1024;
// Cost of a block: a two-tile block keeps the tensor core and the exponentials
// busy for about 3.7k cycles, a one-tile block takes about as long as its
// 64 KB take from HBM on every SM at once, 2.8k.
constexpr int kCostTwo = 4, kCostOne = 3;

struct Sizes {
  int32_t n_ctas;   // CTAs launched
  int32_t B, H_kv, GL;
  int32_t joint;    // 1: no shared items, the prefix belongs to every sequence's items
  int32_t prefix_len, nbp;       // blocks of the prefix
  int32_t groups_p, groups_s;    // row groups of a shared item's key head, of a sequence
  int32_t cost_p, cost_s;        // cost of one block over all those groups
};

__host__ __device__ inline int rows_of(int total, int g) {
  const int r = total - g * kGroup;
  return r < kGroup ? r : kGroup;
}
__host__ __device__ inline int cost_of(int rows) { return rows > 128 ? kCostTwo : kCostOne; }

struct __align__(64) Params {
  CUtensorMap tm_k, tm_v;
  CacheDims c;
  Sizes z;
  int32_t prefix_seq;
  float scale_log2;
  const svg_bf16* q;
  const int32_t *table, *lens, *seqs;
  svg_bf16* o;
  float* lse;
  int* status;
  // workspace
  int32_t* head_item;  // [n_ctas] item that the CTA's piece begins inside of, or -1
  int2* info;          // [items] first CTA and number of pieces
  float* head_o;       // [n_ctas][256][d] piece of the item that began in an earlier CTA
  float2* head_ml;
  float* first_o;      // joint: [n_ctas][256][d]; else [2][rows][d] (shared, own) by q row
  float2* first_ml;
};

struct Barriers {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t o_free, ml_full, drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = 128 * 128;              // 128 rows x 128 B
  static constexpr int kTile = kPanels * kPanel;        // one Q, K or V tile
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffMl = kOffV + kStages * kTile;          // float2 [2][2][128]
  static constexpr int kOffBar = kOffMl + 2 * 2 * 128 * 8;
  static constexpr int kOffBatch = kOffBar + 512;                 // cum, seq, len
  static constexpr int kUsed = kOffBatch + (kMaxBatch + 1) * 8 + 2 * kMaxBatch * 4 + 1024;
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;  // one CTA per SM
  static_assert(sizeof(Barriers) <= 512, "barriers");
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

// Length of entry b's sequence, -1 where the entry is idle, -2 where it is refused.
__device__ __forceinline__ int entry_len(const CacheDims& c, const int32_t* lens, int seq) {
  if (seq < 0) return -1;
  if (seq >= c.max_seqs) return -2;
  const int len = lens[seq];
  return len < 0 || len > c.max_rows() ? -2 : len;
}
__device__ __forceinline__ bool prefix_ok(const CacheDims& c, const int32_t* lens, int seq,
                                          int prefix_len) {
  if (prefix_len == 0) return true;
  const int len = lens[seq];
  return len >= prefix_len && len <= c.max_rows();
}
// Blocks of a sequence's rows after the prefix; block numbers count from row 0
// of the sequence, so the first one may begin before the prefix ends.
__host__ __device__ inline int own_blocks(int len, int prefix_len) {
  return len > prefix_len ? (len + kBK - 1) / kBK - prefix_len / kBK : 0;
}

// A piece of an item: blocks [lo, hi) of its nb.
struct Item {
  int shared, kv, b, g, nb, lo, hi, rows, id;
};

// Walks the items of the cost range [from, to).
struct Walk {
  const Sizes& z;
  const int64_t* cum;  // [B + 1] blocks of the own items before each sequence (one key head, one group)
  int64_t at, from, to;  // cost at which the current item begins
  int shared, kv, b, g;

  __host__ __device__ __forceinline__ int64_t own_cost() const {
    return cum[z.B] * z.cost_s;
  }
  __host__ __device__ Walk(const Sizes& sizes, const int64_t* cum_, int64_t from_, int64_t to_)
      : z(sizes), cum(cum_), from(from_), to(to_) {
    const int64_t per = static_cast<int64_t>(z.nbp) * z.cost_p;
    const int64_t all = z.joint ? 0 : per * z.H_kv;
    int64_t rest = from;
    b = 0;
    if (rest < all) {
      shared = 1;
      kv = static_cast<int>(rest / per);
      rest -= kv * per;
      const int64_t one = static_cast<int64_t>(z.nbp) * kCostTwo;
      g = min(static_cast<int>(rest / one), z.groups_p - 1);
      at = kv * per + g * one;
    } else {
      shared = 0;
      rest -= all;
      const int64_t head = own_cost();
      kv = head > 0 ? static_cast<int>(rest / head) : z.H_kv;
      rest -= kv * head;
      const int64_t blk = rest / z.cost_s;  // the last sequence that begins there
      int lo = 0, hi = z.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= blk) {
          lo = mid;
        } else {
          hi = mid - 1;
        }
      }
      b = lo;
      rest -= cum[b] * z.cost_s;
      const int64_t one = (cum[b + 1] - cum[b]) * kCostTwo;
      g = one > 0 ? min(static_cast<int>(rest / one), z.groups_s - 1) : 0;
      at = all + kv * head + cum[b] * z.cost_s + g * one;
    }
  }
  __host__ __device__ bool next(Item& it) {
    while (at < to && (shared || kv < z.H_kv)) {
      it.shared = shared;
      it.kv = kv;
      it.b = b;
      it.g = g;
      it.nb = shared ? z.nbp : static_cast<int>(cum[b + 1] - cum[b]);
      it.rows = rows_of(shared ? z.B * z.GL : z.GL, g);
      it.id = shared ? kv * z.groups_p + g
                     : (z.joint ? 0 : z.H_kv * z.groups_p) + (kv * z.B + b) * z.groups_s + g;
      const int w = cost_of(it.rows);
      const int64_t begin = at;
      at += static_cast<int64_t>(it.nb) * w;
      // to the next item
      if (shared) {
        if (++g == z.groups_p) {
          g = 0;
          if (++kv == z.H_kv) {
            shared = kv = 0;
          }
        }
      } else if (++g == z.groups_s) {
        g = 0;
        if (++b == z.B) {
          b = 0;
          ++kv;
        }
      }
      it.lo = from > begin ? static_cast<int>((from - begin + w - 1) / w) : 0;
      it.hi = to < at ? static_cast<int>((to - begin + w - 1) / w) : it.nb;
      if (it.lo < it.hi) return true;
    }
    return false;
  }
};

// Where block k of an item lies: block number `blk` of sequence `seq`, of whose
// 128 keys [lo, hi) count.
struct Block {
  int seq, blk, lo, hi;
};
__device__ __forceinline__ Block block_of(const Sizes& z, int prefix_seq, const int* s_seq,
                                          const int* s_len, const Item& it, int k) {
  Block r;
  const int pre = it.shared || z.joint ? z.nbp : 0;
  if (k < pre) {
    r.seq = prefix_seq;
    r.blk = k;
    r.lo = 0;
    r.hi = min(kBK, z.prefix_len - k * kBK);
  } else {
    r.seq = s_seq[it.b];
    r.blk = k - pre + z.prefix_len / kBK;
    r.lo = max(0, z.prefix_len - r.blk * kBK);
    r.hi = min(kBK, s_len[it.b] - r.blk * kBK);
  }
  return r;
}

// q row (and o, lse row) of row r of an item.
__device__ __forceinline__ int64_t q_row(const Sizes& z, const Item& it, int r) {
  r += it.g * kGroup;
  int b = it.b;
  if (it.shared) {
    b = r / z.GL;
    r -= b * z.GL;
  }
  return (static_cast<int64_t>(b) * z.H_kv + it.kv) * z.GL + r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attention_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  Barriers* bar = reinterpret_cast<Barriers*>(smem + C::kOffBar);
  int64_t* s_cum = reinterpret_cast<int64_t*>(smem + C::kOffBatch);
  int* s_seq = reinterpret_cast<int*>(s_cum + kMaxBatch + 1);
  int* s_len = s_seq + kMaxBatch;
  volatile int* abort_flag = &bar->abort_flag;
  const Sizes& z = p.z;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int cta = blockIdx.x;

  // ---- the batch's lengths, and this CTA's piece of the work
  const bool ok_prefix = prefix_ok(p.c, p.lens, p.prefix_seq, z.prefix_len);
  for (int b = tid; b < z.B; b += kThreads) {
    const int seq = p.seqs[b];
    const int len = entry_len(p.c, p.lens, seq);
    if (cta == 0 && (len == -2 || !ok_prefix)) atomicOr(p.status, kDevErrBounds);
    s_seq[b] = seq;
    s_len[b] = len;
    s_cum[b + 1] = len < 0 || !ok_prefix ? 0
                                         : own_blocks(len, z.prefix_len) + (z.joint ? z.nbp : 0);
  }
  __syncthreads();
  if (warp == 0) {
    int64_t sum = 0;
    for (int b0 = 0; b0 < z.B; b0 += 32) {
      int64_t x = b0 + tid < z.B ? s_cum[b0 + tid + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      x += sum;
      if (b0 + tid < z.B) s_cum[b0 + tid + 1] = x;
      sum = __shfl_sync(0xffffffffu, x, 31);
    }
    if (tid == 0) s_cum[0] = 0;
  }
  __syncthreads();
  int64_t total = s_cum[z.B] * z.cost_s * z.H_kv;
  if (!z.joint && ok_prefix) total += static_cast<int64_t>(z.nbp) * z.cost_p * z.H_kv;
  // No piece is smaller than a block, so that every CTA from an item's first to
  // its last has a piece of it.
  const int64_t most = total / kCostTwo < 1 ? 1 : total / kCostTwo;
  const int n_pieces = static_cast<int>(most < z.n_ctas ? most : z.n_ctas);
  if (cta >= n_pieces || total == 0) {
    if (tid == 0) p.head_item[cta] = -1;
    return;
  }
  const int64_t from = total * cta / n_pieces, to = total * (cta + 1) / n_pieces;

  // ---- barriers and tensor memory
  if (warp == 0) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (tid == 32) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->q_full[s], kLoadThreads);
      mbar_init(&bar->q_empty[s], 1);
      mbar_init(&bar->s_full[s], 1);
      mbar_init(&bar->p_full[s], 128);
      mbar_init(&bar->o_final[s], 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
    }
    mbar_init(&bar->o_free, 256);
    mbar_init(&bar->ml_full, 256);
    mbar_init(&bar->drain, 1);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  Walk walk(z, s_cum, from, to);
  Item it;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kProducerWarp) {
      // ---------------------------------------------------------- producer
      // A block is 128 / box boxes of min(page_size, 128) rows, times the panels;
      // a lane loads one of them. Boxes without a row that counts and pages
      // past the pool are read from past the end of the map: zeros.
      const int lane = lane_id();
      const int box = min(p.c.ps, kBK);
      const int boxes = kBK / box;
      const int bx = lane % boxes, pn = lane / boxes;
      const bool loads = pn < C::kPanels;
      const int past = p.c.n_pages * p.c.H_kv * p.c.ps;
      auto page_of = [&](const Block& blk) {  // -1: no row of this lane's box counts
        if (!loads || bx * box >= blk.hi || (bx + 1) * box <= blk.lo) return -1;
        const int page = __ldg(p.table + static_cast<int64_t>(blk.seq) * p.c.max_pages +
                               (blk.blk * kBK + bx * box) / p.c.ps);
        if (page >= 0 && page < p.c.n_pages) return page;
        atomicOr(p.status, kDevErrBounds);
        return -1;
      };
      int n = 0;  // blocks issued
      bool ok = true;
      while (ok && walk.next(it)) {
        Block blk = block_of(z, p.prefix_seq, s_seq, s_len, it, it.lo);
        int page = page_of(blk);
        for (int k = it.lo; k < it.hi; ++k, ++n) {
          const int y = page < 0 ? past
                                 : (page * p.c.H_kv + it.kv) * p.c.ps +
                                       (blk.blk * kBK + bx * box) % p.c.ps;
          if (k + 1 < it.hi) {  // the next block's pages, while this one waits
            blk = block_of(z, p.prefix_seq, s_seq, s_len, it, k + 1);
            page = page_of(blk);
          }
          const int st = n % C::kStages;
          const uint32_t par = ((n / C::kStages) & 1) ^ 1;
          if (lane == 0) {
            ok = mbar_wait(&bar->k_empty[st], par, abort_flag, p.status);
            if (ok) mbar_arrive_expect_tx(&bar->k_full[st], C::kTile);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (loads)
            tma_load_3d(sK + st * C::kTile + pn * C::kPanel + bx * box * 128, &p.tm_k,
                        &bar->k_full[st], pn * 64, y, 0);
          if (lane == 0) {
            ok = mbar_wait(&bar->v_empty[st], par, abort_flag, p.status);
            if (ok) mbar_arrive_expect_tx(&bar->v_full[st], C::kTile);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            ++n;  // the keys of this block are on their way
            break;
          }
          if (loads)
            tma_load_3d(sV + st * C::kTile + pn * C::kPanel + bx * box * 128, &p.tm_v,
                        &bar->v_full[st], pn * 64, y, 0);
        }
      }
      if (!ok && lane == 0) {
        // Let every copy this warp started land before the CTA retires; a
        // barrier that nothing was posted on just runs into the limit.
        for (int j = (n > C::kStages ? n - C::kStages : 0); j < n; ++j) {
          const int st = j % C::kStages;
          const uint32_t par = (j / C::kStages) & 1;
          const long long t0 = clock64();
          while (!(mbar_try_wait(&bar->k_full[st], par) && mbar_try_wait(&bar->v_full[st], par)) &&
                 clock64() - t0 < kWaitLimitCycles) {
          }
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      if (lane_id() == 0) {
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kBK, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
        const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
        int n0 = 0, qn = 0, items = 0;
        uint32_t pp = 0;  // bit t: parity of the next P of softmax warpgroup t
        bool ok = true;
        auto qk = [&](int t, int slot, int st) {
          const uint32_t a0 = q_addr + slot * C::kTile, b0 = k_addr + st * C::kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::kPanel + (kk & 3) * 32;
            mma_bf16_ss(tmem + t * 256, sdesc_sw128(a0 + off, 16, 1024),
                        sdesc_sw128(b0 + off, 16, 1024), idesc_qk, kk > 0 ? 1u : 0u);
          }
          tc_commit(&bar->s_full[t]);
        };
        auto pv = [&](int t, int st, bool first) {
          const uint32_t b0 = v_addr + st * C::kTile;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma_bf16_ts(tmem + t * 256 + 128, tmem + t * 256 + kk * 8,
                        sdesc_sw128(b0 + kk * 16 * 128, C::kPanel, 1024), idesc_pv,
                        (!first || kk > 0) ? 1u : 0u);
        };
        auto wait_p = [&](int t) {
          ok = ok && mbar_wait(&bar->p_full[t], (pp >> t) & 1u, abort_flag, p.status);
          pp ^= 1u << t;
          return ok;
        };
        auto wait = [&](uint64_t* b, uint32_t parity) {
          if (ok) ok = mbar_wait(b, parity, abort_flag, p.status);
          return ok;
        };
        while (ok && walk.next(it)) {
          const int n = it.hi - it.lo;
          const bool two = it.rows > 128;
          for (int t = 0; t < (two ? 2 : 1); ++t)
            wait(&bar->q_full[(qn + t) & 1], ((qn + t) >> 1) & 1);
          if (!ok) break;
          for (int j = 0; ok && j <= n; ++j) {
            const int st = (n0 + j) % C::kStages, par = ((n0 + j) / C::kStages) & 1;
            const int pst = (n0 + j - 1 + C::kStages) % C::kStages;
            const int ppar = ((n0 + j - 1) / C::kStages) & 1;
            if (j == 1 && items > 0 && !wait(&bar->o_free, (items - 1) & 1)) break;
            if (two) {
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if (j > 0) {
                  if (t == 0 && !wait(&bar->v_full[pst], ppar)) break;
                  if (!wait_p(t)) break;
                  tc_fence_after();
                  pv(t, pst, j == 1);
                  if (j == n) tc_commit(&bar->o_final[t]);
                }
                if (j < n) {
                  if (t == 0 && !wait(&bar->k_full[st], par)) break;
                  tc_fence_after();
                  qk(t, (qn + t) & 1, st);
                  if (j == n - 1) tc_commit(&bar->q_empty[(qn + t) & 1]);
                }
              }
              if (!ok) break;
              if (j > 0) tc_commit(&bar->v_empty[pst]);
              if (j < n) tc_commit(&bar->k_empty[st]);
            } else {
              if (j < n) {
                if (!wait(&bar->k_full[st], par)) break;
                tc_fence_after();
                qk(j & 1, qn & 1, st);
                tc_commit(&bar->k_empty[st]);
                if (j == n - 1) tc_commit(&bar->q_empty[qn & 1]);
              }
              if (j > 0) {
                const int t = (j - 1) & 1;
                if (!wait(&bar->v_full[pst], ppar)) break;
                if (!wait_p(t)) break;
                tc_fence_after();
                pv(t, pst, j <= 2);
                tc_commit(&bar->v_empty[pst]);
                if (j >= n - 1) tc_commit(&bar->o_final[t]);  // the tile's last block
              }
            }
          }
          n0 += n;
          qn += two ? 2 : 1;
          ++items;
        }
        if (!ok) {
          // Retire every MMA issued so far before tensor memory is released.
          tc_commit(&bar->drain);
          const long long t0 = clock64();
          while (!mbar_try_wait(&bar->drain, 0) && clock64() - t0 < kWaitLimitCycles) {
          }
        }
      }
    } else {
      // ---------------------------------------------------------- query rows
      const int lt = tid - (kMmaWarp + 1) * 32;
      constexpr int kVecs = D / 8;  // 16-byte vectors of a row
      const uint32_t q_addr = smem_u32(sQ);
      const int vec = lt % kVecs;
      int qn = 0;
      bool ok = true;
      while (ok && walk.next(it)) {
        for (int r0 = 0; r0 < it.rows; r0 += 128, ++qn) {
          ok = mbar_wait(&bar->q_empty[qn & 1], ((qn >> 1) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          const uint32_t dst = q_addr + (qn & 1) * C::kTile + (vec >> 3) * C::kPanel;
          const int rows = min(it.rows - r0, 128);
          for (int r = lt / kVecs; r < rows; r += kLoadThreads / kVecs)
            cp_async16(dst + r * 128 + (((vec & 7) ^ (r & 7)) << 4),
                       p.q + q_row(z, it, r0 + r) * D + vec * 8);
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();
          mbar_arrive(&bar->q_full[qn & 1]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax (tile t)
    const int t = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lanes + t * 256, o_col = s_col + 128;
    int n0 = 0, sc = 0, ones = 0;
    uint32_t fp = 0;  // bit t: parity of the next final commit of tile t
    bool ok = true;
    if (tid == 0) p.head_item[cta] = -1;
    while (ok && walk.next(it)) {
      const int n = it.hi - it.lo;
      const bool two = it.rows > 128;
      const int rows = two ? min(max(it.rows - t * 128, 0), 128) : it.rows;
      const bool active = (warp & 3) * 32 < rows;  // warp-uniform
      float m = -INFINITY, l = 0.0f;                // log2 units
      for (int j = two ? 0 : t; j < n; j += two ? 1 : 2, ++sc) {
        const Block blk = block_of(z, p.prefix_seq, s_seq, s_len, it, it.lo + j);
        const bool ragged = blk.lo > 0 || blk.hi < kBK;
        ok = mbar_wait(&bar->s_full[t], sc & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          uint32_t sr[kBK];
#pragma unroll
          for (int ch = 0; ch < kBK / 32; ++ch)
            tmem_ld_32x32b_x32(s_col + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
          tmem_ld_wait();
          reg_fence(sr);
          if (ragged) {
#pragma unroll
            for (int i = 0; i < kBK; ++i)
              if (i < blk.lo || i >= blk.hi) sr[i] = __float_as_uint(-INFINITY);
          }
          float xm[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) xm[c] = fmaxf(u2f(sr[2 * c]), u2f(sr[2 * c + 1]));
#pragma unroll
          for (int i = 16; i < kBK; i += 16) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              xm[c] = fmax3(xm[c], u2f(sr[i + 2 * c]), u2f(sr[i + 2 * c + 1]));
          }
          const float m_tile =
              fmaxf(fmax3(xm[0], xm[1], xm[2]), fmax3(xm[3], fmax3(xm[4], xm[5], xm[6]), xm[7])) *
              p.scale_log2;
          const bool rebase = m_tile > m + kRebaseLog2;
          const float m_new = rebase ? m_tile : m;
          const float alpha = rebase ? fast_exp2(m - m_new) : 1.0f;
          const float m_use = m_new == -INFINITY ? 0.0f : m_new;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int ch = 0; ch < kBK / 32; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c0 = ch * 32 + 2 * i;
              float y0, y1;
              ffma2(y0, y1, u2f(sr[c0]), u2f(sr[c0 + 1]), p.scale_log2, p.scale_log2, -m_use,
                    -m_use);
              const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
              fadd2(s0, s1, s0, s1, e0, e1);
              pk[i] = pack_bf16x2(e0, e1);
            }
            tmem_st_32x32b_x16(s_col + ch * 16, pk);
          }
          l = l * alpha + (s0 + s1);
          m = m_new;
          tmem_st_wait();
          // This tile's previous PV retired with the commit of this S.
          if (j >= (two ? 1 : 2) && __any_sync(0xffffffffu, rebase)) {
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_col + ch * 32, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(u2f(o[i]) * alpha);
              tmem_st_32x32b_x32(o_col + ch * 32, o);
            }
            tmem_st_wait();
          }
        }
        // Values that do not count may hold anything; a weight of 0 times NaN is
        // NaN, so their rows are cleared before the product reads them (with two
        // tiles by the first one's threads: its product comes first).
        if (ragged && (!two || t == 0)) {
          const int st = (n0 + j) % C::kStages;
          ok = mbar_wait(&bar->v_full[st], ((n0 + j) / C::kStages) & 1, abort_flag, p.status);
          if (!ok) break;
          if (r < blk.lo || r >= blk.hi) {
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn) {
              uint4* row = reinterpret_cast<uint4*>(sV + st * C::kTile + pn * C::kPanel + r * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&bar->p_full[t]);
      }
      if (!ok) break;

      // ---- epilogue
      const bool whole = it.lo == 0 && it.hi == it.nb;
      const bool final_rows = z.joint && whole;
      float fa = 1.0f, fb = 0.0f;  // weights of the two tiles' O (one-tile items)
      const bool both = !two && n > 1;
      if (!two) {
        float2* ml = s_ml + (ones & 1) * 256;
        ml[t * 128 + r] = make_float2(m, l);
        mbar_arrive(&bar->ml_full);
        ok = mbar_wait(&bar->ml_full, ones & 1, abort_flag, p.status);
        if (!ok) break;
        ++ones;
        const float2 a = ml[r], b = ml[128 + r];
        m = fmaxf(a.x, b.x);
        const float m_use = m == -INFINITY ? 0.0f : m;
        fa = fast_exp2(a.x - m_use);
        fb = fast_exp2(b.x - m_use);
        l = a.y * fa + b.y * fb;
      }
      // every thread counts the final commits of both tiles
      if (two) {
        ok = mbar_wait(&bar->o_final[t], (fp >> t) & 1u, abort_flag, p.status);
        fp ^= 3u;
      } else {
        ok = mbar_wait(&bar->o_final[0], fp & 1u, abort_flag, p.status);
        if (ok && both) ok = mbar_wait(&bar->o_final[1], fp >> 1, abort_flag, p.status);
        fp ^= both ? 3u : 1u;
      }
      if (!ok) break;
      tc_fence_after();
      const int rr = two ? t * 128 + r : r;  // row of the item
      const bool valid = r < rows;
      const int64_t row = valid ? q_row(z, it, rr) : 0;
      const int64_t slot = static_cast<int64_t>(cta) * kGroup + rr;
      float* out = nullptr;
      float2* out_ml = nullptr;
      if (it.lo > 0) {
        out = p.head_o + slot * D;
        out_ml = p.head_ml + slot;
      } else if (z.joint) {
        out = p.first_o + slot * D;
        out_ml = p.first_ml + slot;
      } else {
        const int64_t at = row + (it.shared ? 0 : static_cast<int64_t>(z.B) * z.H_kv * z.GL);
        out = p.first_o + at * D;
        out_ml = p.first_ml + at;
      }
      const float inv_l = l > 0.0f ? 1.0f / l : 0.0f;
      // two tiles: all columns of this tile's O; one tile: this warpgroup's half of both
      const int c_lo = two ? 0 : t * (D / 2), c_n = two ? D : D / 2;
      if (active) {
        for (int c0 = c_lo; c0 < c_lo + c_n; c0 += 32) {
          uint32_t o[32];
          if (two) {
            tmem_ld_32x32b_x32(o_col + c0, o);
            tmem_ld_wait();
            reg_fence(o);
          } else {
            tmem_ld_32x32b_x32(lanes + 128 + c0, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(u2f(o[i]) * fa);
            if (both) {
              uint32_t ob[32];
              tmem_ld_32x32b_x32(lanes + 384 + c0, ob);
              tmem_ld_wait();
              reg_fence(ob);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(u2f(o[i]) + u2f(ob[i]) * fb);
            }
          }
          if (!valid) continue;
          if (final_rows) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = pack_bf16x2(u2f(o[8 * v + 2 * i]) * inv_l, u2f(o[8 * v + 2 * i + 1]) * inv_l);
              dst[v] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(out + c0);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar->o_free);
      if (valid && (two || t == 0)) {
        if (!final_rows) {
          *out_ml = make_float2(m, l);
        } else if (p.lse != nullptr) {
          p.lse[row] = l > 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
      }
      if (tid == 0) {
        if (it.lo > 0) {
          p.head_item[cta] = it.id;
        } else if (!final_rows) {
          // the CTA that has the item's last block
          const int64_t begin = walk.at - static_cast<int64_t>(it.nb) * cost_of(it.rows);
          const int64_t x = begin + static_cast<int64_t>(it.nb - 1) * cost_of(it.rows);
          int64_t last = x * n_pieces / total;
          while (total * (last + 1) / n_pieces <= x) ++last;
          p.info[it.id] = make_int2(cta, static_cast<int>(last) - cta + 1);
        }
      }
      n0 += n;
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- joining the pieces
// A warp of the W that share a row takes every W-th piece, four at a time.
struct Joined {
  float m, l;
};
template <int D>
__device__ __forceinline__ void join_one(float (&o)[D / 32], Joined& s, const float* src, float2 ml) {
  constexpr int kE = D / 32;
  float x[kE];
  const int lane = lane_id();
#pragma unroll
  for (int e = 0; e < kE; ++e) x[e] = src[e * 32 + lane];
  const float m = fmaxf(s.m, ml.x);
  const float m_use = m == -INFINITY ? 0.0f : m;
  const float a = fast_exp2(s.m - m_use), b = fast_exp2(ml.x - m_use);
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = o[e] * a + (ml.x == -INFINITY ? 0.0f : x[e] * b);
  s.l = s.l * a + ml.y * b;
  s.m = m;
}

template <int D>
__device__ __forceinline__ void store_row(const Params& p, int64_t row, const float (&o)[D / 32],
                                          const Joined& s) {
  const float inv = s.l > 0.0f ? 1.0f / s.l : 0.0f;
  const int lane = lane_id();
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    p.o[row * D + e * 32 + lane] = static_cast<svg_bf16>(pack_bf16x2(o[e] * inv, 0.0f) & 0xffffu);
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = s.l > 0.0f ? (s.m + __log2f(s.l)) * 0.69314718055994531f : -INFINITY;
}

// Shared and own items: one row per block of W warps.
template <int D, int W>
__global__ void __launch_bounds__(W * 32) join_rows_kernel(const __grid_constant__ Params p) {
  constexpr int kE = D / 32;
  __shared__ float s_o[W][D];
  __shared__ float2 s_ml[W];
  const Sizes& z = p.z;
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int64_t row = blockIdx.x;
  const int64_t bk = row / z.GL;
  const int b = static_cast<int>(bk / z.H_kv), kv = static_cast<int>(bk % z.H_kv);
  const int rr = static_cast<int>(row % z.GL);
  const int len = entry_len(p.c, p.lens, p.seqs[b]);
  if (len < 0 || !prefix_ok(p.c, p.lens, p.prefix_seq, z.prefix_len)) return;
  float o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.0f;
  Joined s{-INFINITY, 0.0f};
  for (int part = 0; part < 2; ++part) {  // the shared item's pieces, then the own one's
    const int in_item = part == 0 ? b * z.GL + rr : rr;
    if ((part == 0 ? z.nbp : own_blocks(len, z.prefix_len)) == 0) continue;
    const int g = in_item / kGroup;
    const int2 info = p.info[part == 0 ? kv * z.groups_p + g
                                       : z.H_kv * z.groups_p + (kv * z.B + b) * z.groups_s + g];
    const int64_t first = row + (part == 0 ? 0 : static_cast<int64_t>(z.B) * z.H_kv * z.GL);
    const int64_t head = static_cast<int64_t>(info.x) * kGroup + in_item % kGroup;
#pragma unroll 4
    for (int i = warp; i < info.y; i += W) {
      const int64_t at = i == 0 ? first : head + static_cast<int64_t>(i) * kGroup;
      join_one<D>(o, s, (i == 0 ? p.first_o : p.head_o) + at * D,
                  (i == 0 ? p.first_ml : p.head_ml)[at]);
    }
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < kE; ++e) s_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) s_ml[warp] = make_float2(s.m, s.l);
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) join_one<D>(o, s, s_o[w], s_ml[w]);
  }
  store_row<D>(p, row, o, s);
}

// Joint items: block (x, y) joins eight rows of the item that is cut where CTA
// x's piece begins, if that is its first cut; x = 0: rows of sequences without keys.
template <int D>
__global__ void __launch_bounds__(256) join_cuts_kernel(const __grid_constant__ Params p) {
  constexpr int kE = D / 32;
  const Sizes& z = p.z;
  const int warp = threadIdx.x >> 5;
  float o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.0f;
  Joined s{-INFINITY, 0.0f};
  if (!prefix_ok(p.c, p.lens, p.prefix_seq, z.prefix_len)) return;
  if (blockIdx.x == 0) {
    if (z.prefix_len > 0) return;
    const int64_t per = static_cast<int64_t>(z.H_kv) * z.GL;
    for (int b = 0; b < z.B; ++b) {
      if (entry_len(p.c, p.lens, p.seqs[b]) != 0) continue;
      for (int64_t i = blockIdx.y * 8 + warp; i < per; i += gridDim.y * 8)
        store_row<D>(p, b * per + i, o, s);
    }
    return;
  }
  const int cta = blockIdx.x;
  const int id = p.head_item[cta];
  if (id < 0) return;
  const int2 info = p.info[id];
  if (info.x != cta - 1) return;  // an earlier cut's block has it
  Item it;
  it.shared = 0;
  it.g = id % z.groups_s;
  it.b = id / z.groups_s % z.B;
  it.kv = id / z.groups_s / z.B;
  const int r = blockIdx.y * 8 + warp;
  if (r >= rows_of(z.GL, it.g)) return;
  int64_t at = static_cast<int64_t>(info.x) * kGroup + r;
  join_one<D>(o, s, p.first_o + at * D, p.first_ml[at]);
  for (int i = 1; i < info.y; ++i) {
    at += kGroup;
    join_one<D>(o, s, p.head_o + at * D, p.head_ml[at]);
  }
  store_row<D>(p, q_row(z, it, r), o, s);
}

inline int groups(int rows) { return (rows + kGroup - 1) / kGroup; }
inline int group_cost(int rows) {
  const int g = groups(rows);
  return (g - 1) * kCostTwo + cost_of(rows_of(rows, g - 1));
}

// Whether the rows of one sequence fill the row groups so well that gathering
// all sequences' rows over the prefix saves less than a tenth of it.
inline bool joint_by_rows(int B, int GL) {
  return 10.0 * group_cost(B * GL) > 9.0 * static_cast<double>(B) * group_cost(GL);
}

struct Layout {
  size_t info, head_o, head_ml, first_o, first_ml, bytes;
};
Layout layout(const CacheDims& c, int32_t B, int32_t H, int32_t Lq, bool joint) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int GL = H / c.H_kv * Lq;
  const size_t items = static_cast<size_t>(c.H_kv) * B * groups(GL) +
                       (joint ? 0 : static_cast<size_t>(c.H_kv) * groups(B * GL));
  const size_t slots = static_cast<size_t>(kMaxCtas) * kGroup;
  const size_t firsts = joint ? slots : 2 * static_cast<size_t>(B) * H * Lq;
  Layout l;
  l.info = up(kMaxCtas * sizeof(int32_t));
  l.head_o = up(l.info + items * sizeof(int2));
  l.head_ml = up(l.head_o + slots * c.d * sizeof(float));
  l.first_o = up(l.head_ml + slots * sizeof(float2));
  l.first_ml = up(l.first_o + firsts * c.d * sizeof(float));
  l.bytes = up(l.first_ml + firsts * sizeof(float2));
  return l;
}

template <int D>
cudaError_t launch(const Params& p, int64_t rows, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = prefix_attention_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // The register hand-over is only balanced at exactly kLaunchRegs per thread.
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
  kern<<<p.z.n_ctas, kThreads, C::kSmem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.z.joint) {
    join_cuts_kernel<D><<<dim3(p.z.n_ctas, kGroup / 8), 256, 0, stream>>>(p);
  } else {
    join_rows_kernel<D, 4><<<static_cast<unsigned>(rows), 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

size_t prefix_workspace_bytes(const CacheDims& c, int32_t B, int32_t H, int32_t Lq) {
  size_t n = layout(c, B, H, Lq, true).bytes;
  if (!joint_by_rows(B, H / c.H_kv * Lq)) {
    const size_t m = layout(c, B, H, Lq, false).bytes;
    if (m > n) n = m;
  }
  return n;
}

cudaError_t launch_prefix_attention(const PrefixArgs& a, int* status, cudaStream_t stream) {
  Params p;
  memset(&p, 0, sizeof(p));
  const int32_t pool_rows = a.c.n_pages * a.c.H_kv * a.c.ps;
  const int box = a.c.ps < kBK ? a.c.ps : kBK;
  if (!make_tmap_bf16(&p.tm_k, a.k_pages, a.c.d, pool_rows, 1, box) ||
      !make_tmap_bf16(&p.tm_v, a.v_pages, a.c.d, pool_rows, 1, box))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int GL = a.H / a.c.H_kv * a.Lq;
  p.c = a.c;
  p.z.n_ctas = sms < kMaxCtas ? sms : kMaxCtas;
  p.z.B = a.B;
  p.z.H_kv = a.c.H_kv;
  p.z.GL = GL;
  p.z.joint = a.prefix_len == 0 || joint_by_rows(a.B, GL) ? 1 : 0;
  p.z.prefix_len = a.prefix_len;
  p.z.nbp = (a.prefix_len + kBK - 1) / kBK;
  p.z.groups_p = groups(a.B * GL);
  p.z.groups_s = groups(GL);
  p.z.cost_p = group_cost(a.B * GL);
  p.z.cost_s = group_cost(GL);
  p.prefix_seq = a.prefix_seq;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.q = a.q;
  p.table = a.table;
  p.lens = a.lens;
  p.seqs = a.seqs;
  p.o = a.o;
  p.lse = a.lse;
  p.status = status;
  const Layout l = layout(a.c, a.B, a.H, a.Lq, p.z.joint != 0);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.head_item = reinterpret_cast<int32_t*>(ws);
  p.info = reinterpret_cast<int2*>(ws + l.info);
  p.head_o = reinterpret_cast<float*>(ws + l.head_o);
  p.head_ml = reinterpret_cast<float2*>(ws + l.head_ml);
  p.first_o = reinterpret_cast<float*>(ws + l.first_o);
  p.first_ml = reinterpret_cast<float2*>(ws + l.first_ml);
  const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.Lq;
  return a.c.d == 128 ? launch<128>(p, rows, stream) : launch<64>(p, rows, stream);
}

}  // namespace svg
