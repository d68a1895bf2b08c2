// How svg_prefix_attention's work is cut into pieces, one or a few for each CTA: what is
// decided on the host (the form of a call, the sizes of a kernel's line) and what each CTA finds
// by itself from the lengths, which only the device knows. Integers alone, the same on host and
// device: prefix_attention.cu says what the items and the line of cost are.
#pragma once

#include <cstring>

#include "internal.h"

namespace svg {
namespace prefix {

constexpr int kBK = 128;             // keys of a block
constexpr int kGroup = 256;          // rows of an item
constexpr int kMaxCtas = 148;
constexpr int kMaxBatch = 1024;
constexpr int kMaxRounds = 16;       // in which items are dealt out
constexpr int kFewRows = 16;    // rows of an item of the few-row kernel
constexpr int kFewWarps = 4;    // that compute
// Cost of a block: a two-tile block takes 3.4k to 3.7k cycles of products and
// exponentials at either head width. A one-tile block takes at d = 128 about as long as its
// 64 KB take from HBM on every SM at once, 2.8k; at d = 64, with 32 KB, less: 32 rows over 60000
// shared rows, 24 heads, 76 blocks a CTA, take 132 us at d = 128 and 91 us at d = 64 (3.3k
// and 2.3k cycles a block, beginning and end of the call included). The units are those of
// d = 128 for both: at d = 64 a one-tile block costs up to a third less than they say.
constexpr int kCostTwo = 4, kCostOne = 3;

// Keys of a block of the few-row kernel.
__host__ __device__ constexpr int few_block(int d) { return kFewWarps * 2048 / d; }

// CTAs of a kernel on a device (or a share of one) with `sms` SMs: one each, but two at least, since
// the two kernels of a mixed batch share them out and none may be left with no CTA. CTAs do not wait
// for one another, so they need not be resident together.
__host__ __device__ inline int ctas_of(int sms) {
  return sms < 2 ? 2 : sms > kMaxCtas ? kMaxCtas : sms;
}

struct Sizes {
  int32_t n_ctas;   // CTAs launched
  int32_t B, H_kv, GL;
  int32_t group;    // most rows of an item
  int32_t shared, own;           // which items there are
  int32_t joint;    // 1: no shared items, the prefix belongs to every sequence's own items
  int32_t prefix_len, nbp;       // blocks of the prefix
  int32_t groups_p, groups_s;    // row groups of a shared item's key head, of a sequence
  int32_t cost_p, cost_s;        // cost of one block over all those groups
  int64_t shared_cost;           // of all shared items, also where another kernel has them
  int32_t shared_items;          // of the tile kernel
  int32_t mixed;                 // 1: the other kind of items is another kernel's, at the same time
};

__host__ __device__ inline int rows_of(int total, int g, int group) {
  const int r = total - g * group;
  return r < group ? r : group;
}
__host__ __device__ inline int cost_of(int rows) { return rows > 128 ? kCostTwo : kCostOne; }

__host__ __device__ inline int least(int a, int b) { return a < b ? a : b; }

// Blocks of `bk` keys of a sequence's rows after the prefix; block numbers count
// from row 0 of the sequence, so the first one may begin before the prefix ends.
__host__ __device__ inline int own_blocks(int len, int prefix_len, int bk) {
  return len > prefix_len ? (len + bk - 1) / bk - prefix_len / bk : 0;
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

  __host__ __device__ Walk(const Sizes& sizes, const int64_t* cum_) : z(sizes), cum(cum_) {}

  __host__ __device__ inline int64_t own_cost() const {
    return z.own ? cum[z.B] * z.cost_s : 0;
  }
  __host__ __device__ void start(int64_t from_, int64_t to_) {
    from = from_;
    to = to_;
    const int64_t per = static_cast<int64_t>(z.nbp) * z.cost_p;
    const int64_t all = z.shared ? per * z.H_kv : 0;
    int64_t rest = from;
    b = 0;
    if (rest < all) {
      shared = 1;
      kv = static_cast<int>(rest / per);
      rest -= kv * per;
      const int64_t one = static_cast<int64_t>(z.nbp) * kCostTwo;
      g = least(static_cast<int>(rest / one), z.groups_p - 1);
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
      g = one > 0 ? least(static_cast<int>(rest / one), z.groups_s - 1) : 0;
      at = all + kv * head + cum[b] * z.cost_s + g * one;
    }
  }
  __host__ __device__ bool next(Item& it) {
    while (at < to && (shared || (z.own && kv < z.H_kv))) {
      it.shared = shared;
      it.kv = kv;
      it.b = b;
      it.g = g;
      it.nb = shared ? z.nbp : static_cast<int>(cum[b + 1] - cum[b]);
      it.rows = rows_of(shared ? z.B * z.GL : z.GL, g, z.group);
      it.id = shared ? kv * z.groups_p + g : (kv * z.B + b) * z.groups_s + g;
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

// Cost at which item i begins, in the order of the walk (those without blocks counted).
__host__ __device__ inline int64_t item_begin(const Sizes& z, const int64_t* cum, int64_t i) {
  const int64_t per = z.shared ? static_cast<int64_t>(z.nbp) * z.cost_p : 0;
  const int shared = z.shared ? z.H_kv * z.groups_p : 0;
  if (i < shared) {
    const int kv = static_cast<int>(i) / z.groups_p, g = static_cast<int>(i) - kv * z.groups_p;
    return kv * per + static_cast<int64_t>(g) * z.nbp * kCostTwo;
  }
  const int j = static_cast<int>(i - shared), pair = j / z.groups_s, g = j - pair * z.groups_s;
  const int kv = pair / z.B, b = pair - kv * z.B;
  return per * z.H_kv + (kv * cum[z.B] + cum[b]) * z.cost_s +
         g * (cum[b + 1] - cum[b]) * kCostTwo;
}

// How the line is cut. First `rounds` times n_pieces items are dealt out whole, one in
// turn to each CTA, so that at any time the CTAs are at neighbouring items, which read the
// same keys, and those come from L2. The rest is cut so that all CTAs have the same in all.
// No piece is smaller than a block, so that every CTA from an item's first to
// its last has a piece of it. 3600 rows of two sequences over 7200 and 3600 rows, 24
// heads, d = 128: one cut line reads 3.2 GB from HBM (L2 gives 35 %) and takes 1075 us, with
// 4 rounds dealt 0.23 GB (89 %) and 929 us, most of it for the clock, which the
// power of those reads held down. At kMaxRounds the items are so short that what all CTAs
// have of the line at a time stays in L2 anyway.
struct Cuts {
  int64_t total;
  int n_pieces, rounds;
  const int64_t* at;  // [n_pieces + 1] where the pieces of the rest begin, with rounds
  __host__ __device__ inline int64_t begin(int w) const {
    return rounds ? at[w] : total * w / n_pieces;
  }
};
// Rounds of a line whose largest item costs `most`: each CTA has a block left at least.
__host__ __device__ inline int deal_rounds(int64_t total, int n, int64_t most) {
  const int64_t r = (total / n - kCostTwo) / most;
  return r < 0 ? 0 : r > kMaxRounds ? kMaxRounds : static_cast<int>(r);
}
__host__ __device__ inline int64_t rest_begin(const Sizes& z, const int64_t* cum, const Cuts& c, int w) {
  int64_t before = 0;  // cost dealt to the CTAs before this one
  for (int j = 0; j < c.rounds; ++j) {
    const int64_t i = static_cast<int64_t>(j) * c.n_pieces;
    before += item_begin(z, cum, i + w) - item_begin(z, cum, i);
  }
  return item_begin(z, cum, static_cast<int64_t>(c.rounds) * c.n_pieces) + c.total * w / c.n_pieces -
         before;
}

// SMs that the few-row kernel takes of n while the tile kernel has the rest: as the time of
// their work. In units of the tile kernel's cost (0.5 us): one of the few-row kernel's blocks 3/2,
// an item's beginning and end 1, one of the tile kernel's items 8 beside its blocks. Both
// kernels are launched with n CTAs and those past their share leave at once, since the
// lengths are not known on the host. At d = 128, one kernel after the other and side by
// side: rows of 64 sequences over 20001 shared rows and up to 700 of their own, four
// query heads to a key head, 79 and 59 us; of 40 over 20000 and 64, 24 heads, 82 and 70 us.
// (Without the tile kernel's items: rows of 150 over 700 and up to 30, eight heads to a key
// head, 54 us instead of 47.)
// With the few-row kernel's work taken for 1/2, 2/3, 1, 4/3 and 2 times as much, in us: at d = 128 the
// first of these calls 70 61 59 69 79, the second 101 84 71 71 76; at d = 64 the first 65 56 50 53
// 59, the second 119 89 68 55 54, rows of 100 over 3000 and up to 200, two heads to a key head,
// 48 44 41 47 59. No one share is the best at d = 64; the second call would want more of the SMs.
__host__ __device__ inline int few_share(int n, int64_t blocks, int64_t items, int64_t tile_cost,
                                         int tile_items) {
  if (blocks == 0) return 0;
  const int64_t few = 3 * blocks + 2 * items;
  const int64_t s = n * few / (few + 2 * (tile_cost + 8 * tile_items));
  return s < 1 ? 1 : s > n - 1 ? n - 1 : static_cast<int>(s);
}

// Cuts the line of a kernel. cum[B + 1]: sequences with own items; cum[B + 2] (read with `deal`): blocks
// of the longest. `shared`: z.shared_cost, or 0 where the prefix is refused. False: there is
// nothing. With rounds the caller then sets at[0 .. n_pieces] to rest_begin.
__host__ __device__ inline bool cut_line(const Sizes& z, const int64_t* cum, int64_t shared, bool deal,
                                         Cuts& cuts) {
  const int64_t own = cum[z.B] * z.H_kv;  // blocks, of one group of rows each
  int n = z.n_ctas;
  if (z.mixed) {
    const int few = few_share(n, own, cum[z.B + 1] * z.H_kv, shared, z.shared_items);
    n = z.own ? few : n - few;
  }
  cuts.total = (z.own ? own * z.cost_s : 0) + (z.shared ? shared : 0);
  cuts.rounds = 0;
  if (cuts.total == 0) return false;
  const int64_t blocks = cuts.total / kCostTwo < 1 ? 1 : cuts.total / kCostTwo;
  cuts.n_pieces = blocks < n ? static_cast<int>(blocks) : n;
  if (deal) {
    const int64_t most_own = z.own ? cum[z.B + 2] : 0;
    const int64_t most = z.shared && shared > 0 && z.nbp > most_own ? z.nbp : most_own;
    cuts.rounds = deal_rounds(cuts.total, n, most * kCostTwo);
  }
  return true;
}

// Number of pieces of the item whose first block CTA `cta` has; it ends at `end`.
__host__ __device__ inline int pieces_of(const Item& it, int64_t end, const Cuts& cuts, int cta) {
  const int64_t x = end - cost_of(it.rows);  // where the last block begins
  int last = cuts.rounds ? cta : static_cast<int>(x * cuts.n_pieces / cuts.total);
  while (cuts.begin(last + 1) <= x) ++last;
  return last - cta + 1;
}

// The costs between which round `j` of CTA `cta` lies; the last one is its piece of the rest.
__host__ __device__ inline longlong2 round_range(const Sizes& z, const int64_t* cum, const Cuts& cuts,
                                                 int cta, int j) {
  if (j == cuts.rounds) return make_longlong2(cuts.begin(cta), cuts.begin(cta + 1));
  const int64_t i = static_cast<int64_t>(j) * cuts.n_pieces + cta;
  return make_longlong2(item_begin(z, cum, i), item_begin(z, cum, i + 1));
}

inline int groups(int rows, int group) { return (rows + group - 1) / group; }
inline int group_cost(int rows, int group) {
  const int g = groups(rows, group);
  return (g - 1) * kCostTwo + cost_of(rows_of(rows, g - 1, group));
}

// Which kernel has which items. Rows of one sequence up to 16 (what a tile of mma.sync
// holds): its own keys go to the few-row kernel, and the prefix too if all sequences' rows are up
// to 16. Otherwise joint items, unless gathering all sequences' rows over the
// prefix saves a tenth of it or more.
// The same calls with the few-row kernel / with the tile kernel in its place, in us, at d = 64; at
// d = 128 (query rows to a key head: 1, then 16):
//   a prefix alone, 60000 rows, 24 heads          64 / 89, 64 / 88;    115 / 122, 117 / 132
//   a prefix of 20001 and up to 700 own rows,     39 / 79, 106 / 192;  49 / 80, 112 / 182
//     64 sequences, 8 key heads
//   2000 to 3000 own rows after one shared row,   108 / 184, 117 / 176;  194 / 230, 284 / 252
//     60 sequences, 16 key heads
// so that 16 rows are right but for long rows of their own at d = 128.
enum Form { kFew, kMixed, kGathered, kJoint };
inline Form form_of(int B, int GL, bool prefix) {
  if (GL <= kFewRows) return B * GL <= kFewRows || !prefix ? kFew : kMixed;
  if (!prefix) return kJoint;
  return 10.0 * group_cost(B * GL, kGroup) > 9.0 * static_cast<double>(B) * group_cost(GL, kGroup)
             ? kJoint
             : kGathered;
}

// The sizes of one kernel's line: the few-row kernel's or the tile kernel's.
inline Sizes sizes_of(int B, int H_kv, int GL, int d, int prefix_len, int n_ctas, bool few,
                      Form form) {
  const int bk = few ? few_block(d) : kBK, group = few ? kFewRows : kGroup;
  Sizes z;
  memset(&z, 0, sizeof(z));
  z.n_ctas = n_ctas;
  z.B = B;
  z.H_kv = H_kv;
  z.GL = GL;
  z.group = group;
  z.mixed = form == kMixed;
  z.shared = prefix_len > 0 && form != kJoint && !(few && form == kMixed);
  z.own = few || form != kMixed;
  z.joint = form == kJoint;
  z.prefix_len = prefix_len;
  z.nbp = (prefix_len + bk - 1) / bk;
  z.groups_p = groups(B * GL, group);
  z.groups_s = groups(GL, group);
  z.cost_p = group_cost(B * GL, group);
  z.cost_s = group_cost(GL, group);
  // the tile kernel's, but where the few-row kernel has all
  z.shared_items = H_kv * groups(B * GL, kGroup);
  z.shared_cost = form == kFew ? static_cast<int64_t>(z.nbp) * z.cost_p * z.H_kv
                               : static_cast<int64_t>((prefix_len + kBK - 1) / kBK) *
                                     group_cost(B * GL, kGroup) * z.H_kv;
  return z;
}

}  // namespace prefix
}  // namespace svg
