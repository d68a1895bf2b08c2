// Attention of a batch of sequences over the history they share and each
// one's own rows after it, keys and values read from cache pages.
//
// O_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i), s = scale q.k: one
// pass over the keys with a running maximum and sum per row. Two disjoint key
// sets give (O, m, l) each, joined exactly by
//   m = max(m1, m2), l = sum l_k 2^(m_k - m), O = sum O_k 2^(m_k - m) / l,
// which is what makes the work divisible along the keys. A NaN score leaves the
// maximum alone (a maximum skips NaN) and makes l and O NaN, and nothing after it takes them
// for anything else: "no key" is l = 0, not a maximum of -inf, which a row of NaN has too.
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
// fp32 and joined by a second kernel. Where there are several items to a CTA, whole
// ones are dealt out first and only the rest is cut (see Cuts).
//
// One CTA per SM walks its piece. 384 threads: warps 0-3 and 4-7 softmax
// and epilogue (thread = row = tensor-memory lane), warp 8 loads K, warp 9 issues
// the products, warp 10 loads V, warp 11 query rows (K and V apart, since a V
// buffer is free only after its softmax, and the K after it must not wait for that).
// Two forms of an item:
//   two tiles  129..256 rows: tile A and tile B, each block serves both;
//   one tile   up to 128 rows: tile A and tile B hold the SAME rows, A takes
//              the even blocks and B the odd ones, so that one's softmax
//              overlaps the other's products, and the two are joined in the epilogue.
// Tensor memory holds S and O of both tiles; P (bf16) overwrites S at d = 128. The
// weights are rounded to bf16 because the tensor core multiplies them with bf16 values
// (off by at most 2^-8 of each); row sums are taken before that rounding, in
// fp32, as are the maxima and O.
//
// Measured: 3600 rows of two sequences over 7200 shared and 3600 own rows, 24 heads,
// d = 128 (956 GFLOP): 929 us, 1029 TFLOP/s, a two-tile block in 3.6k cycles of which the
// products take 2.05k if nothing holds them up (Q K^T reads both operands from shared
// memory, at some 100 cycles instead of 64; the softmax of a tile takes 1.9k).
// 1020 rows of three over 4080 and up to 2100 rows, 48 heads, d = 64 (212 GFLOP): 368 us; a
// block's exponentials alone take 2.05k cycles of its 3.7k. A CTA needs some 14k cycles before
// its first products (lengths and pages in turn, code not yet in the caches) and 5k for its
// last piece's (O, m, l), which is what small calls cost.
#include <cstring>

#include "internal.h"
#include "prefix_line.h"
#include "sm100.cuh"

namespace svg {
namespace {

using namespace prefix;

constexpr int kThreads = 384;
constexpr int kKWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kVWarp = 10;
constexpr int kLaunchRegs = 168;
constexpr int kSoftmaxRegs = 216;
constexpr int kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * kLaunchRegs, "register split");
constexpr float kRebaseLog2 = 8.0f;  // O is re-based when a maximum grows by more than 2^8

// Where the pieces of one kind of items (shared or own) go: a slot holds
// `stride` rows, row r's channels 4c .. 4c + 3 as a float4 at r * rs + c * cs. The tile
// kernel, with a row per lane, writes slots channel by channel (rs = 1), the
// few-row kernel row by row (cs = 1), so that either writes whole lines.
struct Pieces {
  int2* info;       // [items] first CTA and number of pieces
  float4* first_o;  // pieces with an item's first block: a slot per item, or (joint) per CTA
  float2* first_ml;
  float4* head_o;   // piece of the item that began in an earlier CTA: a slot per CTA
  float2* head_ml;
  int32_t stride, rs, cs;
  int32_t group;    // rows of an item at most
  int32_t groups;   // items of a key head (shared) or of a sequence and key head (own)
};

struct __align__(64) Params {
  CUtensorMap tm_k, tm_v;
  CUtensorMap tm_q, tm_q_rows;  // the rows of q in boxes of 128, for items of one sequence, and one by one
  CacheDims c;
  Sizes z;
  int32_t prefix_seq;
  float scale_log2;
  const svg_bf16 *q, *k_pages, *v_pages;
  const int32_t *table, *lens, *seqs;
  svg_bf16* o;
  float* lse;
  int* status;
  // workspace
  int32_t* head_item;  // joint: [n_ctas] item that the CTA's piece begins inside of, or -1
  Pieces part[2];      // shared, own
};

// What the roles of a CTA need to know of a piece of an item, in shared memory: the
// query-row warp walks the line of cost, the others read.
struct __align__(16) Order {
  int shared, kv, rows;
  int lo, hi, nb;         // blocks [lo, hi) of nb; hi = 0: no more items
  int pre, hi_pre;        // the first `pre` blocks are the prefix's, the last of which has hi_pre keys
  int lo_own, hi_last;    // keys that count of the first block after them begin at lo_own, of the
                          // last one end at hi_last
  int seq, blk0;          // its sequence, and the number there of the first block after the prefix
  int row0;               // first q row (items of one sequence)
  int id, pieces;         // number, and pieces it is cut into
  int unused;
};
constexpr int kOrders = 4;

// A reader's place in the ring of orders.
struct Orders {
  Order* ring;
  uint64_t *full, *empty;
  volatile int* abort_flag;
  int* status;
  int n = 0;
  // The next order; false: there is none (or a wait ran out). Every lane of the warp calls it.
  __device__ __forceinline__ bool take(Order& it) {
    if (!mbar_wait(&full[n % kOrders], (n / kOrders) & 1, abort_flag, status)) return false;
    it = ring[n % kOrders];
    __syncwarp();
    if (it.hi == 0) return false;
    if (lane_id() == 0) mbar_arrive(&empty[n % kOrders]);
    ++n;
    return true;
  }
};

struct Barriers {
  uint64_t item_full[kOrders], item_empty[kOrders];
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_final[2];
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
  // Tensor memory. At d = 64 there is room for P beside S: the next S = Q K^T of a
  // tile then starts as soon as its S is in registers, and not after P V.
  static constexpr bool kOwnP = D == 64;
  static __device__ __forceinline__ uint32_t col_s(int t) { return t * (kOwnP ? 128 : 256); }
  static __device__ __forceinline__ uint32_t col_p(int t) { return kOwnP ? 256 + t * 64 : col_s(t); }
  static __device__ __forceinline__ uint32_t col_o(int t) {
    return kOwnP ? 384 + t * 64 : 128 + t * 256;
  }
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffMl = kOffV + kStages * kTile;          // float2 [2][2][128]
  static constexpr int kOffBar = kOffMl + 2 * 2 * 128 * 8;
  static constexpr int kOffOrder = kOffBar + 512;
  static constexpr int kOffBatch = kOffOrder + kOrders * sizeof(Order);  // cum, cuts, rounds, seq, len
  static constexpr int kUsed = kOffBatch + (kMaxBatch + 4 + kMaxCtas + 2 + 2 * (kMaxRounds + 1)) * 8 +
                               2 * kMaxBatch * 4 + 1024;
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;  // one CTA per SM
  static_assert(sizeof(Barriers) <= 512, "barriers");
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

struct FewBarriers {
  uint64_t item_full[kOrders], item_empty[kOrders];
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
  uint64_t sync;
  int abort_flag;
};

template <int D>
struct FewCfg {
  static constexpr int kKeys = few_block(D) / kFewWarps;  // keys of a block that a warp takes
  static constexpr int kBlock = few_block(D);      // kFewWarps times that
  static constexpr int kPanel = kBlock * 128;
  static constexpr int kTile = D / 64 * kPanel;    // 16 KB
  static constexpr int kStages = 4;
  static constexpr int kQRow = D * 2 + 16;         // bytes from row to row: no bank conflicts
  static constexpr int kORow = D + 8;              // floats, likewise
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffO = kOffV + kStages * kTile;  // float [2][warps][16][kORow], by turns
  static constexpr int kOffMl = kOffO + 2 * kFewWarps * kFewRows * kORow * 4;
  static constexpr int kOffQ = kOffMl + 2 * kFewWarps * kFewRows * 8;
  static constexpr int kOffBar = kOffQ + 2 * kFewRows * kQRow;
  static constexpr int kOffOrder = kOffBar + 512;
  static constexpr int kOffBatch = kOffOrder + kOrders * sizeof(Order);
  static constexpr int kSmem = kOffBatch + (kMaxBatch + 3) * 8 + 2 * kMaxBatch * 4 + 1024;
  static_assert(sizeof(FewBarriers) <= 512, "barriers");
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

// 1 / l and the natural log-sum-exp of a row with maximum m (log2 units) and sum l. No weight
// at all is O = 0, lse = -inf; NaN stays NaN.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

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
// q row (and o, lse row) of row r of an item.
__device__ __forceinline__ int64_t q_row(const Sizes& z, const Item& it, int r) {
  r += it.g * z.group;
  int b = it.b;
  if (it.shared) {
    b = r / z.GL;
    r -= b * z.GL;
  }
  return (static_cast<int64_t>(b) * z.H_kv + it.kv) * z.GL + r;
}

// The batch's lengths into shared memory and the cuts of the line of cost; false: this CTA
// has no piece. Every CTA finds the same line. `s_at`: room for the cuts of a line
// that is dealt.
template <int T, int BK, int FEW_BK, bool DEAL>
__device__ __forceinline__ bool plan_pieces(const Params& p, int64_t* s_cum, int* s_seq, int* s_len,
                                            int64_t* s_at, Cuts& cuts) {
  const Sizes& z = p.z;
  const int tid = threadIdx.x, cta = blockIdx.x;
  const bool ok_prefix = prefix_ok(p.c, p.lens, p.prefix_seq, z.prefix_len);
  for (int b = tid; b < z.B; b += T) {
    const int seq = p.seqs[b];
    const int len = entry_len(p.c, p.lens, seq);
    if (cta == 0 && (len == -2 || !ok_prefix)) atomicOr(p.status, kDevErrBounds);
    s_seq[b] = seq;
    s_len[b] = len;
    s_cum[b + 1] = len < 0 || !ok_prefix
                       ? 0
                       : own_blocks(len, z.prefix_len, z.own ? BK : FEW_BK) + (z.joint ? z.nbp : 0);
  }
  __syncthreads();
  if (tid < 32) {
    int64_t sum = 0;
    int some = 0;  // sequences with blocks
    int most = 0;  // blocks of one
    for (int b0 = 0; b0 < z.B; b0 += 32) {
      int64_t x = b0 + tid < z.B ? s_cum[b0 + tid + 1] : 0;
      some += __popc(__ballot_sync(0xffffffffu, x > 0));
      most = max(most, static_cast<int>(x));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      x += sum;
      if (b0 + tid < z.B) s_cum[b0 + tid + 1] = x;
      sum = __shfl_sync(0xffffffffu, x, 31);
    }
    if (DEAL) most = __reduce_max_sync(0xffffffffu, most);
    if (tid == 0) {
      s_cum[0] = 0;
      s_cum[z.B + 1] = some;
      if (DEAL) s_cum[z.B + 2] = most;
    }
  }
  __syncthreads();
  cuts.at = s_at;
  if (!cut_line(z, s_cum, ok_prefix ? z.shared_cost : 0, DEAL, cuts)) return false;
  if (DEAL && cuts.rounds > 0) {
    for (int w = tid; w <= cuts.n_pieces; w += T) s_at[w] = rest_begin(z, s_cum, cuts, w);
    __syncthreads();
  }
  return cta < cuts.n_pieces;
}

// One arrival for a warp's 32: arrivals on one address are taken one by one.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The role of a warp that loads K or V: the blocks of every order, through a ring of
// STAGES tiles of BK rows x D / 64 panels. A block is BK / box boxes of
// min(page_size, BK) rows, times the panels; a lane loads one of them. Boxes without
// a row that counts and pages past the pool are read from past the end of
// the map: zeros.
template <int D, int BK, int STAGES>
__device__ __forceinline__ void stream_blocks(const Params& p, const CUtensorMap* map, uint8_t* ring,
                                              uint64_t* full, uint64_t* empty, Orders& orders) {
  constexpr int kPanels = D / 64, kPanel = BK * 128, kTile = kPanels * kPanel;
  const int lane = lane_id();
  const int box = min(p.c.ps, BK);
  const int boxes = BK / box;
  const int bx = lane % boxes, pn = lane / boxes;
  const bool loads = pn < kPanels;
  const int past = p.c.n_pages * p.c.H_kv * p.c.ps;
  Order it = {};
  // 64 consecutive page numbers of a sequence, lane i the i-th of either half; the second
  // half is on its way while the first is used, so that only an item's first block waits
  // for the table (a load of it takes as long as a block's share of HBM).
  int w_seq = -1, w_base = 0, w0 = 0, w1 = 0;
  auto page_at = [&](int seq, int i) {
    return i < p.c.max_pages ? __ldg(p.table + static_cast<int64_t>(seq) * p.c.max_pages + i) : -1;
  };
  // row of the pool that this lane's box of block k begins at
  auto row_of = [&](int k) {
    const bool own = k >= it.pre;
    const int lo = k == it.pre ? it.lo_own : 0;
    const int hi = k == it.pre - 1 ? it.hi_pre : own && k == it.nb - 1 ? it.hi_last : BK;
    const int seq = own ? it.seq : p.prefix_seq;
    const int pos0 = (own ? k - it.pre + it.blk0 : k) * BK;
    const int first = pos0 / p.c.ps, pos = pos0 + bx * box;
    if (seq != w_seq || first < w_base || first >= w_base + 64) {
      w_seq = seq;
      w_base = first;
      w0 = page_at(seq, first + lane);
      w1 = page_at(seq, first + 32 + lane);
    } else if (first >= w_base + 32) {
      w_base += 32;
      w0 = w1;
      w1 = page_at(seq, w_base + 32 + lane);
    }
    const int at = loads ? pos / p.c.ps - w_base : 0;  // at most 7 past `first`
    const int p0 = __shfl_sync(0xffffffffu, w0, at & 31), p1 = __shfl_sync(0xffffffffu, w1, at & 31);
    if (!loads || bx * box >= hi || (bx + 1) * box <= lo) return past;
    const int page = at < 32 ? p0 : p1;
    if (page >= 0 && page < p.c.n_pages)
      return (page * p.c.H_kv + it.kv) * p.c.ps + pos % p.c.ps;
    atomicOr(p.status, kDevErrBounds);
    return past;
  };
  int n = 0;  // blocks issued
  bool ok = true;
  while (ok && orders.take(it)) {
    for (int k = it.lo; k < it.hi; ++k, ++n) {
      const int y = row_of(k);
      const int st = n % STAGES;
      if (lane == 0) {
        ok = mbar_wait(&empty[st], ((n / STAGES) & 1) ^ 1, orders.abort_flag, p.status);
        if (ok) mbar_arrive_expect_tx(&full[st], kTile);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (loads)
        tma_load_3d(ring + st * kTile + pn * kPanel + bx * box * 128, map, &full[st], pn * 64, y, 0);
    }
  }
  if (*orders.abort_flag && lane == 0) {
    // Let every copy this warp started land before the CTA retires.
    for (int j = (n > STAGES ? n - STAGES : 0); j < n; ++j) {
      const long long t0 = clock64();
      while (!mbar_try_wait(&full[j % STAGES], (j / STAGES) & 1) &&
             clock64() - t0 < kWaitLimitCycles) {
      }
    }
  }
}

// The next item of the walk as an order (none: the end), for the warp that publishes
// them. False: a wait ran out.
template <int BK>
__device__ __forceinline__ bool publish(const Params& p, Orders& orders, bool more, const Item& item,
                                        int pieces, const int* s_seq, const int* s_len) {
  const Sizes& z = p.z;
  const int at = orders.n % kOrders;
  const bool ok = mbar_wait(&orders.empty[at], ((orders.n / kOrders) & 1) ^ 1, orders.abort_flag,
                            p.status);
  if (!__all_sync(0xffffffffu, ok)) return false;
  if (lane_id() == 0) {
    Order w;
    memset(&w, 0, sizeof(w));
    if (more) {
      w.shared = item.shared;
      w.kv = item.kv;
      w.rows = item.rows;
      w.lo = item.lo;
      w.hi = item.hi;
      w.nb = item.nb;
      w.pre = item.shared || z.joint ? z.nbp : 0;
      w.hi_pre = z.prefix_len - (z.nbp - 1) * BK;
      w.lo_own = z.prefix_len % BK;
      w.blk0 = z.prefix_len / BK;
      if (!item.shared) {
        w.seq = s_seq[item.b];
        w.hi_last = s_len[item.b] - (w.blk0 + item.nb - w.pre - 1) * BK;
        w.row0 = static_cast<int>(q_row(z, item, 0));
      }
      w.id = item.id;
      w.pieces = pieces;
    }
    orders.ring[at] = w;
    mbar_arrive(&orders.full[at]);
  }
  ++orders.n;
  return true;
}

// DEAL: there are more items than CTAs, so that some may be dealt out whole. A kernel of its
// own, since with that code in it the others took 1.5 us longer to get going.
template <int D, bool DEAL>
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
  Order* s_order = reinterpret_cast<Order*>(smem + C::kOffOrder);
  int64_t* s_cum = reinterpret_cast<int64_t*>(smem + C::kOffBatch);
  int64_t* s_at = s_cum + kMaxBatch + 4;
  longlong2* s_range = reinterpret_cast<longlong2*>(s_at + kMaxCtas + 2);
  int* s_seq = reinterpret_cast<int*>(s_range + kMaxRounds + 1);
  int* s_len = s_seq + kMaxBatch;
  volatile int* abort_flag = &bar->abort_flag;
  const Sizes& z = p.z;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int cta = blockIdx.x;
  launch_dependents();  // the join waits for this kernel's end by itself
  if (tid == 0) {
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
    prefetch_tensormap(z.shared ? &p.tm_q_rows : &p.tm_q);
  }

  Cuts cuts;
  if (!plan_pieces<kThreads, kBK, FewCfg<D>::kBlock, DEAL>(p, s_cum, s_seq, s_len, s_at, cuts)) {
    if (z.joint && tid == 0) p.head_item[cta] = -1;
    if (tid == 0) wait_for_primary();
    return;
  }
  if (DEAL && tid <= cuts.rounds) s_range[tid] = round_range(z, s_cum, cuts, cta, tid);

  // ---- barriers and tensor memory
  if (warp == 0) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (tid == 32) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->q_full[s], 1);
      mbar_init(&bar->q_empty[s], 1);
      mbar_init(&bar->s_full[s], 1);
      mbar_init(&bar->s_free[s], 4);  // warps
      mbar_init(&bar->p_full[s], 4);
      mbar_init(&bar->pv_done[s], 1);
      mbar_init(&bar->o_final[s], 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
    }
    for (int s = 0; s < kOrders; ++s) {
      mbar_init(&bar->item_full[s], 1);
      mbar_init(&bar->item_empty[s], 11);  // K, V and MMA warps, eight softmax warps
    }
    mbar_init(&bar->o_free, 8);
    mbar_init(&bar->ml_full, 8);
    mbar_init(&bar->drain, 1);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  Orders orders{s_order, bar->item_full, bar->item_empty, abort_flag, p.status};
  Order it = {};
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kKWarp || warp == kVWarp) {
      const bool is_k = warp == kKWarp;
      stream_blocks<D, kBK, C::kStages>(p, is_k ? &p.tm_k : &p.tm_v, is_k ? sK : sV,
                                        is_k ? bar->k_full : bar->v_full,
                                        is_k ? bar->k_empty : bar->v_empty, orders);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs this, so that what the products take (descriptors,
      // addresses) is uniform; one lane issues them.
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kBK, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
      const bool on = elect_one();
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV), C::kPanel, 1024);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      int n0 = 0, qn = 0, items = 0;  // blocks, query tiles, items so far
      uint32_t pp = 0;                // bit t: parity of the next P of softmax warpgroup t
      uint32_t sf = 3;                // bit t: parity of tile t's last but one reading of S
      bool ok = true;
      auto qk = [&](int t, int slot, int st) {
        const uint64_t a = q_desc + slot * (C::kTile >> 4), b = k_desc + st * (C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int kUnit = 16;
          const int off = ((kk >> 2) * C::kPanel + (kk & 3) * 32) / kUnit;
          mma_bf16_ss_on(on, tm + C::col_s(t), a + off, b + off, idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit_on(on, &bar->s_full[t]);
      };
      auto pv = [&](int t, int st, bool first) {
        const uint64_t b = v_desc + st * (C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          mma_bf16_ts_on(on, tm + C::col_o(t), tm + C::col_p(t) + kk * 8, b + kk * 128, idesc_pv,
                         (!first || kk > 0) ? 1u : 0u);
        if (C::kOwnP) tc_commit_on(on, &bar->pv_done[t]);
      };
      auto ready = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test(b, parity)) != 0;
      };
      while (orders.take(it)) {
        const int n = __shfl_sync(0xffffffffu, it.hi - it.lo, 0);
        const bool two = __shfl_sync(0xffffffffu, it.rows, 0) > 128;
        if (!C::kOwnP && two) {
          // P is where S was, so a tile's Q K^T follows its P V anyway: P V and Q K^T of one
          // tile, then of the other.
          auto wait = [&](uint64_t* b, uint32_t parity) {
            ok = ok && mbar_wait(b, parity, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok) != 0;
            return ok;
          };
          for (int j = 0; j <= n; ++j) {
            const int st = (n0 + j) % C::kStages, vst = (n0 + j + C::kStages - 1) % C::kStages;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (j > 0) {
                if (t == 0 && !wait(&bar->v_full[vst], ((n0 + j - 1) / C::kStages) & 1)) break;
                if (t == 0 && j == 1 && items > 0 && !wait(&bar->o_free, (items - 1) & 1)) break;
                if (!wait(&bar->p_full[t], (pp >> t) & 1u)) break;
                pp ^= 1u << t;
                tc_fence_after();
                pv(t, vst, j == 1);
                if (t == 1) tc_commit_on(on, &bar->v_empty[vst]);
                if (j == n) tc_commit_on(on, &bar->o_final[t]);
              }
              if (j < n) {
                if (j == 0 && !wait(&bar->q_full[(qn + t) & 1], ((qn + t) >> 1) & 1)) break;
                if (t == 0 && !wait(&bar->k_full[st], ((n0 + j) / C::kStages) & 1)) break;
                tc_fence_after();
                qk(t, (qn + t) & 1, st);
                if (t == 1) tc_commit_on(on, &bar->k_empty[st]);
                if (j == n - 1) tc_commit_on(on, &bar->q_empty[(qn + t) & 1]);
              }
            }
            if (!ok) break;
          }
          if (!ok) break;
          n0 += n;
          qn += 2;
          ++items;
          continue;
        }
        // The products that may come next (two tiles, Q K^T or P V) are issued as
        // their operands get ready; in a fixed order one tile waits for what
        // the other's softmax has still to do. With one tile of rows tile 1 has the odd
        // blocks. S of a tile is overwritten once it was read (P apart) or after its
        // P V (products complete in the order of issue).
        const int step = two ? 1 : 2;
        int q[2] = {0, two ? 0 : 1}, v[2] = {0, two ? 0 : 1};  // next block of each
        long long idle = 0;                                    // since when nothing was ready
        while (v[0] < n || v[1] < n) {
          bool did = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int vst = (n0 + v[t]) % C::kStages, kst = (n0 + q[t]) % C::kStages;
            if (v[t] < q[t] && v[t] < n && ready(&bar->p_full[t], (pp >> t) & 1u) &&
                ready(&bar->v_full[vst], ((n0 + v[t]) / C::kStages) & 1) &&
                (v[t] >= step || items == 0 || ready(&bar->o_free, (items - 1) & 1))) {
              tc_fence_after();
              pv(t, vst, v[t] < step);
              pp ^= 1u << t;
              v[t] += step;
              if (!two || v[1 - t] >= v[t]) tc_commit_on(on, &bar->v_empty[vst]);
              if (v[t] >= n) tc_commit_on(on, &bar->o_final[t]);
              did = true;
            }
            const int slot = (qn + (two ? t : 0)) & 1;
            if (q[t] < n && (C::kOwnP ? ready(&bar->s_free[t], (sf >> t) & 1u) : v[t] == q[t]) &&
                ready(&bar->k_full[kst], ((n0 + q[t]) / C::kStages) & 1) &&
                (q[t] >= step || ready(&bar->q_full[slot], ((qn + (two ? t : 0)) >> 1) & 1))) {
              tc_fence_after();
              qk(t, slot, kst);
              sf ^= 1u << t;
              q[t] += step;
              if (!two || q[1 - t] >= q[t]) tc_commit_on(on, &bar->k_empty[kst]);
              if (q[t] >= n && (two || q[1 - t] >= n)) tc_commit_on(on, &bar->q_empty[slot]);
              did = true;
            }
          }
          if (did) {
            idle = 0;
          } else if (idle == 0) {
            idle = clock64();
          } else if (__any_sync(0xffffffffu,
                                *abort_flag || clock64() - idle > kWaitLimitCycles)) {
            if (!*abort_flag && on) atomicOr(p.status, kDevErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
        }
        if (!ok) break;
        n0 += n;
        qn += two ? 2 : 1;
        ++items;
      }
      if (*abort_flag) {
        // Retire every MMA issued so far before tensor memory is released.
        tc_commit_on(on, &bar->drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(&bar->drain, 0) && clock64() - t0 < kWaitLimitCycles) {
        }
      }
    } else {
      // ---------------------------------------------------------- query rows
      // The rows of one sequence are one run of q: a tiled load (what it brings of
      // other rows past the item's end is never used). The rows of several are
      // gathered, four to a lane. (Copied by cp.async to the same places, 64 to a lane, they
      // took 5k cycles a tile, in which nothing else can begin.)
      const int lane = lane_id();
      int qn = 0;
      bool ok = true;
      Walk walk(z, s_cum);
      Item item;
      int round = DEAL ? -1 : 0;
      if constexpr (!DEAL) walk.start(cuts.begin(cta), cuts.begin(cta + 1));
      for (bool more = true; more;) {
        if constexpr (DEAL) {
          while (round < 0 || !walk.next(item)) {
            more = ++round <= cuts.rounds;
            if (!more) break;
            walk.start(s_range[round].x, s_range[round].y);
          }
        } else {
          more = walk.next(item);
        }
        const int pieces = !more || item.lo > 0 ? 0
                           : round < cuts.rounds ? 1 : pieces_of(item, walk.at, cuts, cta);
        if (!publish<kBK>(p, orders, more, item, pieces, s_seq, s_len)) break;
        if (!more) break;
        for (int r0 = 0; r0 < item.rows; r0 += 128, ++qn) {
          uint64_t* full = &bar->q_full[qn & 1];
          ok = mbar_wait(&bar->q_empty[qn & 1], ((qn >> 1) & 1) ^ 1, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = more = false;
            break;
          }
          uint8_t* dst = sQ + (qn & 1) * C::kTile;
          if (!item.shared) {
            if (lane == 0) {
              const int64_t row = q_row(z, item, r0);
              mbar_arrive_expect_tx(full, C::kTile);
              for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_3d(dst + pn * C::kPanel, &p.tm_q, full, pn * 64, static_cast<int>(row), 0);
            }
            continue;
          }
          const int fours = (min(item.rows - r0, 128) + 3) / 4;
          if (lane == 0) mbar_arrive_expect_tx(full, fours * 4 * 128 * C::kPanels);
          __syncwarp();
          if (lane < fours) {
            int row[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)  // past the item's end its last row again, not used
              row[i] = static_cast<int>(q_row(z, item, min(r0 + 4 * lane + i, item.rows - 1)));
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
              tma_gather4(dst + pn * C::kPanel + lane * 512, &p.tm_q_rows, full, pn * 64, row[0],
                          row[1], row[2], row[3]);
          }
        }
      }
      if (*abort_flag && lane == 0) {
        // Let the loads this warp started land before the CTA retires.
        for (int j = (qn > 2 ? qn - 2 : 0); j < qn; ++j) {
          const long long t0 = clock64();
          while (!mbar_try_wait(&bar->q_full[j & 1], (j >> 1) & 1) &&
                 clock64() - t0 < kWaitLimitCycles) {
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax (tile t)
    const int t = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lanes + C::col_s(t), p_col = lanes + C::col_p(t);
    const uint32_t o_col = lanes + C::col_o(t);
    int n0 = 0, sc = 0, ones = 0;
    uint32_t fp = 0;  // bit t: parity of the next final commit of tile t
    bool ok = true;
    if (z.joint && tid == 0) p.head_item[cta] = -1;
    while (ok && orders.take(it)) {
      const int n = it.hi - it.lo;
      const bool two = it.rows > 128;
      const int rows = two ? min(max(it.rows - t * 128, 0), 128) : it.rows;
      const bool active = (warp & 3) * 32 < rows;  // warp-uniform
      float m = -INFINITY, l = 0.0f;                // log2 units
      for (int j = two ? 0 : t; j < n; j += two ? 1 : 2, ++sc) {
        const int k = it.lo + j;
        const int k_lo = k == it.pre ? it.lo_own : 0;  // the keys of this block that count
        const int k_hi =
            k == it.pre - 1 ? it.hi_pre : k >= it.pre && k == it.nb - 1 ? it.hi_last : kBK;
        const bool ragged = k_lo > 0 || k_hi < kBK;
        ok = mbar_wait(&bar->s_full[t], sc & 1, abort_flag, p.status);
        if (!ok) break;
        __syncwarp();
        tc_fence_after();
        uint32_t sr[kBK];
        if (active) {
#pragma unroll
          for (int ch = 0; ch < kBK / 32; ++ch)
            tmem_ld_32x32b_x32(s_col + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
          tmem_ld_wait();
          reg_fence(sr);
        }
        if (C::kOwnP) {
          tc_fence_before();
          warp_arrive(&bar->s_free[t]);
        }
        if (active) {
          if (ragged) {
#pragma unroll
            for (int i = 0; i < kBK; ++i)
              if (i < k_lo || i >= k_hi) sr[i] = __float_as_uint(-INFINITY);
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
          // P and O are free again once the previous block's product is done
          if (C::kOwnP && sc > 0) {
            ok = mbar_wait(&bar->pv_done[t], (sc - 1) & 1, abort_flag, p.status);
            __syncwarp();
            tc_fence_after();
          }
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
            tmem_st_32x32b_x16(p_col + ch * 16, pk);
          }
          l = l * alpha + (s0 + s1);
          m = m_new;
          tmem_st_wait();
          // This tile's previous PV has retired: with the commit of this S, or waited for.
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
        // A warp without rows waits for that product too: its arrival for this block
        // must not be taken for one for the previous block, whose P may still be on its way.
        if (C::kOwnP && !active && sc > 0)
          ok = mbar_wait(&bar->pv_done[t], (sc - 1) & 1, abort_flag, p.status);
        // Values that do not count may hold anything; a weight of 0 times NaN is
        // NaN, so their rows are cleared before the product reads them (by
        // both tiles' threads: either product may come first).
        if (ragged) {
          const int st = (n0 + j) % C::kStages;
          ok = mbar_wait(&bar->v_full[st], ((n0 + j) / C::kStages) & 1, abort_flag, p.status);
          if (!ok) break;
          if (r < k_lo || r >= k_hi) {
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
        warp_arrive(&bar->p_full[t]);
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
        warp_arrive(&bar->ml_full);
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
      __syncwarp();
      tc_fence_after();
      const int rr = two ? t * 128 + r : r;  // row of the item
      const bool valid = r < rows;
      const int64_t row = it.row0 + rr;
      const Pieces& part = p.part[it.shared ? 0 : 1];
      const int64_t slot =
          static_cast<int64_t>(it.lo > 0 || z.joint ? cta : it.id) * part.stride;
      float4* out = (it.lo > 0 ? part.head_o : part.first_o) + slot * (D / 4) + rr;
      float2* out_ml = (it.lo > 0 ? part.head_ml : part.first_ml) + slot + rr;
      const float inv_l = inverse_sum(l);
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
            tmem_ld_32x32b_x32(lanes + C::col_o(0) + c0, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(u2f(o[i]) * fa);
            if (both) {
              uint32_t ob[32];
              tmem_ld_32x32b_x32(lanes + C::col_o(1) + c0, ob);
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
            float4* dst = out + static_cast<int64_t>(c0 / 4) * part.stride;
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v * part.stride] = make_float4(u2f(o[4 * v]), u2f(o[4 * v + 1]),
                                                 u2f(o[4 * v + 2]), u2f(o[4 * v + 3]));
          }
        }
      }
      tc_fence_before();
      warp_arrive(&bar->o_free);
      if (valid && (two || t == 0)) {
        if (!final_rows) {
          *out_ml = make_float2(m, l);
        } else if (p.lse != nullptr) {
          p.lse[row] = log_sum(m, l);
        }
      }
      if (tid == 0) {
        if (it.lo > 0) {
          if (z.joint) p.head_item[cta] = it.id;
        } else if (!final_rows) {
          part.info[it.id] = make_int2(cta, it.pieces);
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
  // This kernel needs nothing of the few-row kernel before it, but the join, which
  // waits for this one, needs both to have ended.
  if (tid == 0) wait_for_primary();
}

// ---------------------------------------------------------------- few rows
// Items of up to 16 rows: one row of a few sequences over a long prefix, or one
// sequence's rows over its own keys. Their products are too small for a
// 128-row tensor-memory tile to pay: its softmax keeps one warp busy (2.1k cycles a
// block) and holds a V buffer meanwhile. What bounds the work is
// reading K and V once. So one CTA per SM streams them through a ring of
// 128 KB, across the borders of items, and four warps take 16 keys (32 at d = 64) of each
// block with mma.sync m16n8k16 (the four joined at the end of a piece):
// a block's 32 KB take 1.4k cycles from HBM, its products and softmax 1.1k of each warp, the
// end of an item 1.8k. One row of 16 sequences over 118800 shared rows, 24 heads,
// d = 128: 241 us for 1.55 GB, 6.4 TB/s; the whole call 248 us, and 374 us with the tile kernel
// in this one's place.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

constexpr int kFewThreads = (kFewWarps + 3) * 32;  // and K, V, and query-row warps

template <int D>
__global__ void __launch_bounds__(kFewThreads, 1) prefix_few_kernel(const __grid_constant__ Params p) {
  using C = FewCfg<D>;
  constexpr int NG = C::kKeys / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FewBarriers* bar = reinterpret_cast<FewBarriers*>(smem + C::kOffBar);
  Order* s_order = reinterpret_cast<Order*>(smem + C::kOffOrder);
  int64_t* s_cum = reinterpret_cast<int64_t*>(smem + C::kOffBatch);
  int* s_seq = reinterpret_cast<int*>(s_cum + kMaxBatch + 3);
  int* s_len = s_seq + kMaxBatch;
  volatile int* abort_flag = &bar->abort_flag;
  const Sizes& z = p.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = lane_id();
  launch_dependents();
  if (tid == 0) {
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
    for (int s = 0; s < kOrders; ++s) {
      mbar_init(&bar->item_full[s], 1);
      mbar_init(&bar->item_empty[s], kFewWarps + 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->q_full[s], 32);
      mbar_init(&bar->q_empty[s], kFewWarps);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], kFewWarps);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], kFewWarps);
    }
    mbar_init(&bar->sync, kFewWarps);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  Cuts cuts;
  if (!plan_pieces<kFewThreads, C::kBlock, C::kBlock, false>(p, s_cum, s_seq, s_len, nullptr, cuts)) return;
  __syncthreads();
  Orders orders{s_order, bar->item_full, bar->item_empty, abort_flag, p.status};

  if (warp == kFewWarps || warp == kFewWarps + 1) {
    const bool is_k = warp == kFewWarps;
    stream_blocks<D, C::kBlock, C::kStages>(p, is_k ? &p.tm_k : &p.tm_v,
                                            smem + (is_k ? C::kOffK : C::kOffV),
                                            is_k ? bar->k_full : bar->v_full,
                                            is_k ? bar->k_empty : bar->v_empty, orders);
    return;
  }
  if (warp == kFewWarps + 2) {
    // ------------------------------------------------------------ orders and query rows
    Walk walk(z, s_cum);
    walk.start(cuts.begin(blockIdx.x), cuts.begin(blockIdx.x + 1));
    Item item;
    for (int qn = 0;; ++qn) {
      const bool more = walk.next(item);
      const int pieces = more && item.lo == 0 ? pieces_of(item, walk.at, cuts, blockIdx.x) : 0;
      if (!publish<C::kBlock>(p, orders, more, item, pieces, s_seq, s_len) || !more) break;
      const bool ok =
          mbar_wait(&bar->q_empty[qn & 1], ((qn >> 1) & 1) ^ 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int mine = lane < item.rows ? static_cast<int>(q_row(z, item, lane)) : 0;
      const uint32_t dst = smem_u32(smem + C::kOffQ + (qn & 1) * kFewRows * C::kQRow);
      constexpr int kVecs = D / 8;
      for (int i = lane / kVecs; i < kFewRows; i += 32 / kVecs) {
        const int src = __shfl_sync(0xffffffffu, mine, i);
        if (i < item.rows)
          cp_async16(dst + i * C::kQRow + (lane % kVecs) * 16,
                     p.q + static_cast<int64_t>(src) * D + (lane % kVecs) * 8);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      mbar_arrive(&bar->q_full[qn & 1]);
    }
    return;
  }

  // -------------------------------------------------------------- products and softmax
  const int w = warp;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t k_addr = smem_u32(smem + C::kOffK), v_addr = smem_u32(smem + C::kOffV);
  // This lane's row of the 8 x 8 matrices of a 16 x 16 tile: K as it lies (key, then the
  // second 8 dims, then the second 8 keys), V to be transposed (second 8 keys first).
  const int k_key = w * C::kKeys + (lane & 7) + (lane >> 4) * 8, k_ch = lane >> 3 & 1;
  const int v_key = w * C::kKeys + (lane & 7) + (lane >> 3 & 1) * 8, v_ch = lane >> 4;
  auto at_of = [](int key, int ch) {  // byte of 16-byte chunk `ch` of a key's row in a swizzled tile
    return (ch >> 3) * C::kPanel + key * 128 + (((ch & 7) ^ (key & 7)) << 4);
  };
  int n0 = 0, items = 0;
  bool ok = true;
  Order it;
  for (; orders.take(it); ++items) {
    uint32_t qa[D / 16][4];  // Q in operand order; rows past the item's hold anything
    ok = mbar_wait(&bar->q_full[items & 1], (items >> 1) & 1, abort_flag, p.status);
    if (!ok) break;
    __syncwarp();
    const uint32_t q_addr = smem_u32(smem + C::kOffQ + (items & 1) * kFewRows * C::kQRow) +
                            ((lane & 7) + (lane >> 3 & 1) * 8) * C::kQRow + (lane >> 4) * 16;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) ldmatrix4(qa[kk], q_addr + kk * 32);
    warp_arrive(&bar->q_empty[items & 1]);

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // rows g and g + 8, log2 units
    for (int k = it.lo; k < it.hi; ++k, ++n0) {
      const int st = n0 % C::kStages, par = (n0 / C::kStages) & 1;
      // keys of this warp's share that count
      const int k_lo = (k == it.pre ? it.lo_own : 0) - w * C::kKeys;
      const int k_hi = (k == it.pre - 1                    ? it.hi_pre
                        : k >= it.pre && k == it.nb - 1 ? it.hi_last
                                                        : C::kBlock) -
                       w * C::kKeys;
      const bool ragged = k_lo > 0 || k_hi < C::kKeys;
      ok = mbar_wait(&bar->k_full[st], par, abort_flag, p.status);
      if (!ok) break;
      __syncwarp();
      // All of K's operands first (with one warp to a scheduler nothing else hides their
      // latency), then the products, in two chains for each 8 keys.
      float s[NG][2][4], s2[NG][2][4];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        uint32_t kb[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ldmatrix4(kb[kk], k_addr + st * C::kTile + at_of(k_key + n * 16, kk * 2 + k_ch));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] = s2[n][u][e] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 2)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_16816(s[n][u], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], kb[kk][2 * u],
                      kb[kk][2 * u + 1]);
            mma_16816(s2[n][u], qa[kk + 1][0], qa[kk + 1][1], qa[kk + 1][2], qa[kk + 1][3],
                      kb[kk + 1][2 * u], kb[kk + 1][2 * u + 1]);
          }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] += s2[n][u][e];
      }
      warp_arrive(&bar->k_empty[st]);
      if (ragged) {
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = n * 16 + u * 8 + 2 * c + (e & 1);
              if (key < k_lo || key >= k_hi) s[n][u][e] = -INFINITY;
            }
      }
      // ---- running maximum and sum of rows g (e = 0, 1) and g + 8 (e = 2, 3)
      float alpha[2], base[2];
      bool rebase = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = -INFINITY;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) x = fmax3(x, s[n][u][2 * r], s[n][u][2 * r + 1]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)) * p.scale_log2;
        const bool up = x > m[r] + kRebaseLog2;
        alpha[r] = up ? fast_exp2(m[r] - x) : 1.0f;
        m[r] = up ? x : m[r];
        base[r] = m[r] == -INFINITY ? 0.0f : m[r];
        rebase = rebase || up;
        l[r] *= alpha[r];
      }
      if (__any_sync(0xffffffffu, rebase)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
      }
      uint32_t pa[NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float e0 = fast_exp2(fmaf(s[n][u][2 * r], p.scale_log2, -base[r]));
            const float e1 = fast_exp2(fmaf(s[n][u][2 * r + 1], p.scale_log2, -base[r]));
            l[r] += e0 + e1;
            pa[n][u * 2 + r] = pack_bf16x2(e0, e1);
          }
      ok = mbar_wait(&bar->v_full[st], par, abort_flag, p.status);
      if (!ok) break;
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        // Values that do not count may hold anything, and 0 times NaN is NaN: cleared.
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of keys 2c, 2c + 1 and 2c + 8, 2c + 9
        if (ragged) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = n * 16 + u * 8 + 2 * c;
            keep[u] = (key >= k_lo && key < k_hi ? 0x0000ffffu : 0u) |
                      (key + 1 >= k_lo && key + 1 < k_hi ? 0xffff0000u : 0u);
          }
        }
        uint32_t vb[D / 16][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          ldmatrix4_trans(vb[i], v_addr + st * C::kTile + at_of(v_key + n * 16, i * 2 + v_ch));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (ragged)
            vb[i][0] &= keep[0], vb[i][1] &= keep[1], vb[i][2] &= keep[0], vb[i][3] &= keep[1];
          mma_16816(o[2 * i], pa[n][0], pa[n][1], pa[n][2], pa[n][3], vb[i][0], vb[i][1]);
          mma_16816(o[2 * i + 1], pa[n][0], pa[n][1], pa[n][2], pa[n][3], vb[i][2], vb[i][3]);
        }
      }
      warp_arrive(&bar->v_empty[st]);
    }
    if (!ok) break;

    // ---- the four warps' (O, m, l) joined; in places by turns, so that one meeting
    // of the warps an item is enough: whoever writes a place again has met
    // the others after they read it
    float* s_o =
        reinterpret_cast<float*>(smem + C::kOffO) + (items & 1) * kFewWarps * kFewRows * C::kORow;
    float2* s_ml = reinterpret_cast<float2*>(smem + C::kOffMl) + (items & 1) * kFewWarps * kFewRows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (g + 8 * r >= it.rows) continue;
      if (c == 0) s_ml[w * kFewRows + g + 8 * r] = make_float2(m[r], l[r]);
      float* dst = s_o + (w * kFewRows + g + 8 * r) * C::kORow + 2 * c;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
    warp_arrive(&bar->sync);
    ok = mbar_wait(&bar->sync, items & 1, abort_flag, p.status);
    if (!ok) break;
    const Pieces& part = p.part[it.shared ? 0 : 1];
    const int64_t slot = static_cast<int64_t>(it.lo > 0 ? blockIdx.x : it.id) * part.stride;
    float4* out = (it.lo > 0 ? part.head_o : part.first_o) + slot * (D / 4);
    float2* out_ml = (it.lo > 0 ? part.head_ml : part.first_ml) + slot;
    for (int i = tid; i < it.rows * (D / 4); i += kFewWarps * 32) {
      const int r = i / (D / 4), ch = i % (D / 4);
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kFewWarps; ++j) top = fmaxf(top, s_ml[j * kFewRows + r].x);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < kFewWarps; ++j) {
        const float2 ml = s_ml[j * kFewRows + r];
        const float f = fast_exp2(ml.x - (top == -INFINITY ? 0.0f : top));
        const float4 y = *reinterpret_cast<const float4*>(s_o + (j * kFewRows + r) * C::kORow + ch * 4);
        x = make_float4(x.x + y.x * f, x.y + y.y * f, x.z + y.z * f, x.w + y.w * f);
        sum += ml.y * f;
      }
      out[i] = x;
      if (ch == 0) out_ml[r] = make_float2(top, sum);
    }
    if (tid == 0 && it.lo == 0) part.info[it.id] = make_int2(blockIdx.x, it.pieces);
    __syncwarp();
  }
}

// ---------------------------------------------------------------- joining the pieces
// A block joins eight rows: lane (r, c) of warp w has row r's float4 number 4w + c,
// which reads either layout of a slot in runs of 64 bytes or more. F warps take
// turns at the pieces of the same channels.
struct Joined {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void join_one(Joined& s, float2 ml, float4 x) {
  const float m = fmaxf(s.m, ml.x);
  const float m_use = m == -INFINITY ? 0.0f : m;
  const float a = fast_exp2(s.m - m_use), b = fast_exp2(ml.x - m_use);
  s.o = make_float4(s.o.x * a + x.x * b, s.o.y * a + x.y * b, s.o.z * a + x.z * b,
                    s.o.w * a + x.w * b);
  s.l = s.l * a + ml.y * b;
  s.m = m;
}

template <int D>
__device__ __forceinline__ void store_row(const Params& p, int64_t row, int c4, const Joined& s) {
  const float inv = inverse_sum(s.l);
  *reinterpret_cast<uint2*>(p.o + row * D + c4 * 4) =
      make_uint2(pack_bf16x2(s.o.x * inv, s.o.y * inv), pack_bf16x2(s.o.z * inv, s.o.w * inv));
  if (p.lse != nullptr && c4 == 0)
    p.lse[row] = log_sum(s.m, s.l);
}

// Pieces k = first, first + step, ... of row r of an item. (A count that cannot be, where a
// kernel gave up before it wrote one, is not followed.)
template <int D>
__device__ __forceinline__ void join_pieces(Joined& s, const Pieces& part, int2 info,
                                            int64_t first_slot, int r, int c4, int first, int step) {
  if (info.x < 0 || info.y < 0 || info.x > kMaxCtas || info.y > kMaxCtas - info.x) return;
#pragma unroll 8
  for (int k = first; k < info.y; k += step) {
    const int64_t slot = (k == 0 ? first_slot : info.x + k) * part.stride;
    join_one(s, (k == 0 ? part.first_ml : part.head_ml)[slot + r],
             (k == 0 ? part.first_o : part.head_o)[slot * (D / 4) + r * part.rs + c4 * part.cs]);
  }
}

// Shared and own items.
template <int D, int F>
__global__ void __launch_bounds__(D * 2 * F) join_rows_kernel(const __grid_constant__ Params p) {
  constexpr int kChunks = D / 16;  // warps that cover a row
  __shared__ float4 s_o[F > 1 ? F - 1 : 1][kChunks * 32];
  __shared__ float2 s_ml[F > 1 ? F - 1 : 1][kChunks * 32];
  const Sizes& z = p.z;
  const int lane = lane_id(), chunk = (threadIdx.x >> 5) % kChunks, f = (threadIdx.x >> 5) / kChunks;
  const int64_t rows = static_cast<int64_t>(z.B) * z.H_kv * z.GL;
  const int64_t row = blockIdx.x * static_cast<int64_t>(8) + (lane >> 2);
  const int c4 = chunk * 4 + (lane & 3);
  Joined s{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  wait_for_primary();
  bool live = row < rows;
  if (live) {
    const int64_t bk = row / z.GL;
    const int rr = static_cast<int>(row - bk * z.GL);
    const int b = static_cast<int>(bk / z.H_kv), kv = static_cast<int>(bk - static_cast<int64_t>(b) * z.H_kv);
    const int len = entry_len(p.c, p.lens, p.seqs[b]);
    live = len >= 0 && prefix_ok(p.c, p.lens, p.prefix_seq, z.prefix_len);
    for (int i = 0; i < 2; ++i) {  // the shared item's pieces, then the own one's
      if (!live || (i == 0 ? z.prefix_len : len - z.prefix_len) <= 0) continue;
      const Pieces& part = p.part[i];
      const int in_item = i == 0 ? b * z.GL + rr : rr;
      const int id = (i == 0 ? kv : kv * z.B + b) * part.groups + in_item / part.group;
      join_pieces<D>(s, part, part.info[id], id, in_item % part.group, c4, f, F);
    }
  }
  if (F > 1) {
    const int at = chunk * 32 + lane;
    if (f > 0) {
      s_o[f - 1][at] = s.o;
      s_ml[f - 1][at] = make_float2(s.m, s.l);
    }
    __syncthreads();
    if (f > 0) return;
#pragma unroll
    for (int i = 0; i < F - 1; ++i) join_one(s, s_ml[i][at], s_o[i][at]);
  }
  if (live) store_row<D>(p, row, c4, s);
}

// Joint items: block (x, y) joins eight rows of the item that is cut where CTA
// x's piece begins, if that is its first cut; x = 0: rows of sequences without keys.
template <int D>
__global__ void __launch_bounds__(D * 2) join_cuts_kernel(const __grid_constant__ Params p) {
  const Sizes& z = p.z;
  const int lane = lane_id();
  const int c4 = (threadIdx.x >> 5) * 4 + (lane & 3);
  Joined s{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  wait_for_primary();
  if (blockIdx.x == 0) {
    if (z.prefix_len > 0) return;
    const int64_t per = static_cast<int64_t>(z.H_kv) * z.GL;
    for (int b = 0; b < z.B; ++b) {
      if (entry_len(p.c, p.lens, p.seqs[b]) != 0) continue;
      for (int64_t i = blockIdx.y * 8 + (lane >> 2); i < per; i += gridDim.y * 8)
        store_row<D>(p, b * per + i, c4, s);
    }
    return;
  }
  const int id = p.head_item[blockIdx.x];
  if (id < 0) return;
  const Pieces& part = p.part[1];
  const int2 info = part.info[id];
  if (info.x != static_cast<int>(blockIdx.x) - 1) return;  // an earlier cut's block has it
  Item it;
  it.shared = 0;
  it.g = id % z.groups_s;
  it.b = id / z.groups_s % z.B;
  it.kv = id / z.groups_s / z.B;
  const int r = blockIdx.y * 8 + (lane >> 2);
  if (r >= rows_of(z.GL, it.g, z.group)) return;
  join_pieces<D>(s, part, info, info.x, r, c4, 0, 1);
  store_row<D>(p, q_row(z, it, r), c4, s);
}

struct Place {
  size_t info, first_o, first_ml, head_o, head_ml;
  int stride, group, groups;
};
struct Layout {
  Place part[2];
  size_t head_item, bytes;
};
Layout layout(const CacheDims& c, int32_t B, int32_t H, int32_t Lq, Form form) {
  const int GL = H / c.H_kv * Lq;
  Layout l;
  memset(&l, 0, sizeof(l));
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) / 256 * 256;
    return here;
  };
  l.head_item = take(kMaxCtas * sizeof(int32_t));
  for (int i = 0; i < 2; ++i) {
    if (i == 0 && (form == kJoint || (form == kFew && B * GL > kFewRows))) continue;  // no shared items
    Place& t = l.part[i];
    const bool few = form == kFew || (form == kMixed && i == 1);
    const int all = i == 0 ? B * GL : GL;
    t.group = few ? kFewRows : kGroup;
    t.groups = groups(all, t.group);
    // tile slots hold whole warps of rows, so that a warp's stores are whole lines
    t.stride = few ? all : all < kGroup ? (all + 31) / 32 * 32 : kGroup;
    const size_t items = static_cast<size_t>(c.H_kv) * (i == 0 ? 1 : B) * t.groups;
    const size_t heads = static_cast<size_t>(kMaxCtas) * t.stride;
    const size_t firsts = form == kJoint ? heads : items * t.stride;
    t.info = take(items * sizeof(int2));
    t.first_o = take(firsts * c.d * sizeof(float));
    t.first_ml = take(firsts * sizeof(float2));
    t.head_o = take(heads * c.d * sizeof(float));
    t.head_ml = take(heads * sizeof(float2));
  }
  l.bytes = at;
  return l;
}

// `after`: behind a kernel of the same call, whose end the kernel waits for itself.
template <typename K>
cudaError_t launch_kernel(K kern, dim3 grid, int threads, int smem, bool after, const Params& p,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, bool DEAL>
cudaError_t launch_tiles(const Params& p, bool after, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = prefix_attention_kernel<D, DEAL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // The register hand-over is only balanced at exactly kLaunchRegs per thread.
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
  return launch_kernel(kern, dim3(p.z.n_ctas), kThreads, C::kSmem, after, p, stream);
}

template <int D>
cudaError_t launch_few(const Params& p, cudaStream_t stream) {
  using C = FewCfg<D>;
  auto kern = prefix_few_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(p.z.n_ctas), kFewThreads, C::kSmem, false, p, stream);
}

// Maps of the pools in boxes of the rows of a page, or of a block where that is less.
bool set_maps(const PrefixArgs& a, Params& p, int bk) {
  const int32_t pool_rows = a.c.n_pages * a.c.H_kv * a.c.ps;
  const int box = a.c.ps < bk ? a.c.ps : bk;
  return make_tmap_bf16(&p.tm_k, a.k_pages, a.c.d, pool_rows, 1, box) &&
         make_tmap_bf16(&p.tm_v, a.v_pages, a.c.d, pool_rows, 1, box);
}

template <int D>
cudaError_t launch(const PrefixArgs& a, Params& p, Form form, int sms, cudaStream_t stream) {
  const int GL = a.H / a.c.H_kv * a.Lq;
  cudaError_t e = cudaSuccess;
  if (form == kFew || form == kMixed) {
    p.z = sizes_of(a.B, a.c.H_kv, GL, a.c.d, a.prefix_len, sms, true, form);
    if (!set_maps(a, p, FewCfg<D>::kBlock)) return cudaErrorInvalidValue;
    if ((e = launch_few<D>(p, stream)) != cudaSuccess) return e;
  }
  if (form != kFew) {
    p.z = sizes_of(a.B, a.c.H_kv, GL, a.c.d, a.prefix_len, sms, false, form);
    if (!set_maps(a, p, kBK) ||
        (p.z.own && !make_tmap_bf16(&p.tm_q, a.q, D, a.B * a.H * a.Lq, 1, 128)) ||
        (p.z.shared &&
         !make_tmap_rows_bf16(&p.tm_q_rows, a.q, D, static_cast<int64_t>(a.B) * a.H * a.Lq)))
      return cudaErrorInvalidValue;
    const int64_t items = static_cast<int64_t>(a.c.H_kv) *
                          ((p.z.shared ? p.z.groups_p : 0) +
                           (p.z.own ? static_cast<int64_t>(a.B) * p.z.groups_s : 0));
    e = items > sms ? launch_tiles<D, true>(p, form == kMixed, stream)
                    : launch_tiles<D, false>(p, form == kMixed, stream);
    if (e != cudaSuccess) return e;
  }
  if (form == kJoint)
    return launch_kernel(join_cuts_kernel<D>, dim3(p.z.n_ctas, kGroup / 8), D * 2, 0, true, p, stream);
  // One row's pieces in turn, or by four warps where there are few rows and so
  // many pieces of each.
  const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.Lq;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (grid >= 148) return launch_kernel(join_rows_kernel<D, 1>, dim3(grid), D * 2, 0, true, p, stream);
  return launch_kernel(join_rows_kernel<D, 4>, dim3(grid), D * 8, 0, true, p, stream);
}

}  // namespace

// What the call itself needs, and what calls of fewer entries or rows might, which another
// form may take: above 2304 rows a sequence the groups are at least nine tenths
// full, so that all calls are joint.
size_t prefix_workspace_bytes(const CacheDims& c, int32_t B, int32_t H, int32_t Lq) {
  const int G = H / c.H_kv, GL = G * Lq;
  size_t most = 0;
  auto take = [&](Form form, int32_t rows) {
    const size_t n = layout(c, B, H, rows, form).bytes;
    if (n > most) most = n;
  };
  if (GL <= kFewRows) {
    take(kFew, Lq);
    take(kMixed, Lq);
  } else {
    take(kJoint, Lq);
    const int rows = 2304 / G < 1 ? 1 : 2304 / G;  // of more heads to a key head one row is more
    take(kGathered, Lq < rows ? Lq : rows);
  }
  take(form_of(B, GL, true), Lq);
  take(form_of(B, GL, false), Lq);
  return most;
}

cudaError_t launch_prefix_attention(const PrefixArgs& a, int* status, cudaStream_t stream) {
  Params p;
  memset(&p, 0, sizeof(p));
  const int GL = a.H / a.c.H_kv * a.Lq;
  const Form form = form_of(a.B, GL, a.prefix_len > 0);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  sms = ctas_of(sms);
  p.c = a.c;
  p.prefix_seq = a.prefix_seq;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.q = a.q;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.table = a.table;
  p.lens = a.lens;
  p.seqs = a.seqs;
  p.o = a.o;
  p.lse = a.lse;
  p.status = status;
  const Layout l = layout(a.c, a.B, a.H, a.Lq, form);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.head_item = reinterpret_cast<int32_t*>(ws + l.head_item);
  for (int i = 0; i < 2; ++i) {
    const bool few = form == kFew || (form == kMixed && i == 1);
    const Place& at = l.part[i];
    Pieces& t = p.part[i];
    t.info = reinterpret_cast<int2*>(ws + at.info);
    t.first_o = reinterpret_cast<float4*>(ws + at.first_o);
    t.first_ml = reinterpret_cast<float2*>(ws + at.first_ml);
    t.head_o = reinterpret_cast<float4*>(ws + at.head_o);
    t.head_ml = reinterpret_cast<float2*>(ws + at.head_ml);
    t.stride = at.stride;
    t.group = at.group;
    t.groups = at.groups;
    t.rs = few ? a.c.d / 4 : 1;
    t.cs = few ? 1 : at.stride;
  }
  return a.c.d == 128 ? launch<128>(a, p, form, sms, stream) : launch<64>(a, p, form, sms, stream);
}

}  // namespace svg
