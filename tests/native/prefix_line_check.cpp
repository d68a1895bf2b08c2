// Walks the pieces of every CTA of one call of svg_prefix_attention on the host, as the kernels
// do, and checks them. Built and called by tests/test_prefix_line.py.
#include <vector>

#include "prefix_line.h"

using namespace svg::prefix;

#define REQUIRE(x)                \
  do {                            \
    if (!(x)) return __LINE__;    \
  } while (0)

namespace {

struct Seen {
  int next = 0, first = -1, n = 0, pieces = 0, nb = 0;
};

// One kernel's line. lens: -1 for an entry without a sequence. out: rounds, pieces.
int check_line(const Sizes& z, int bk, int few_bk, const int* lens, bool ok_prefix, bool deal,
               int* out) {
  std::vector<int64_t> cum(z.B + 3, 0);
  std::vector<int> own(z.B, 0);
  int64_t some = 0, most = 0;
  for (int b = 0; b < z.B; ++b) {
    if (lens[b] >= 0 && ok_prefix)
      own[b] = own_blocks(lens[b], z.prefix_len, z.own ? bk : few_bk) + (z.joint ? z.nbp : 0);
    cum[b + 1] = cum[b] + own[b];
    some += own[b] > 0;
    most = own[b] > most ? own[b] : most;
  }
  cum[z.B + 1] = some;
  cum[z.B + 2] = most;
  Cuts cuts;
  std::vector<int64_t> at(kMaxCtas + 2, -1);
  cuts.at = at.data();
  out[0] = out[1] = 0;
  const int shared_items = z.shared ? z.H_kv * z.groups_p : 0;
  const int own_items = z.own ? z.H_kv * z.B * z.groups_s : 0;
  bool some_work = false;
  for (int b = 0; b < z.B; ++b) some_work = some_work || (z.own && own[b] > 0);
  some_work = some_work || (z.shared && ok_prefix);
  const bool any = cut_line(z, cum.data(), ok_prefix ? z.shared_cost : 0, deal, cuts);
  REQUIRE(any == some_work);
  if (!any) return 0;
  REQUIRE(cuts.n_pieces >= 1 && cuts.n_pieces <= z.n_ctas);
  REQUIRE(cuts.rounds >= 0 && cuts.rounds <= kMaxRounds && (deal || cuts.rounds == 0));
  out[0] = cuts.rounds;
  out[1] = cuts.n_pieces;
  if (cuts.rounds > 0)
    for (int w = 0; w <= cuts.n_pieces; ++w) at[w] = rest_begin(z, cum.data(), cuts, w);
  REQUIRE(cuts.begin(cuts.n_pieces) == cuts.total);

  std::vector<Seen> seen(shared_items + own_items);
  for (int cta = 0; cta < cuts.n_pieces; ++cta) {
    int64_t cost = 0;
    int heads = 0, tails = 0, pieces_of_rest = 0;  // items begun in an earlier CTA, ended in a later one
    for (int round = 0; round <= cuts.rounds; ++round) {
      const longlong2 range = round_range(z, cum.data(), cuts, cta, round);
      REQUIRE(range.x <= range.y && range.x >= 0 && range.y <= cuts.total);
      Walk walk(z, cum.data());
      walk.start(range.x, range.y);
      Item it;
      while (walk.next(it)) {
        REQUIRE(it.lo >= 0 && it.lo < it.hi && it.hi <= it.nb);
        REQUIRE(it.kv >= 0 && it.kv < z.H_kv && it.g >= 0);
        if (it.shared) {
          REQUIRE(z.shared && it.g < z.groups_p && it.nb == z.nbp);
          REQUIRE(it.id == it.kv * z.groups_p + it.g && it.rows == rows_of(z.B * z.GL, it.g, z.group));
        } else {
          REQUIRE(z.own && it.b >= 0 && it.b < z.B && it.g < z.groups_s && it.nb == own[it.b]);
          REQUIRE(it.id == (it.kv * z.B + it.b) * z.groups_s + it.g);
          REQUIRE(it.rows == rows_of(z.GL, it.g, z.group));
        }
        REQUIRE(it.rows >= 1 && it.rows <= z.group);
        if (round < cuts.rounds) {
          REQUIRE(it.lo == 0 && it.hi == it.nb);
        } else {
          ++pieces_of_rest;
        }
        Seen& s = seen[it.shared ? it.id : shared_items + it.id];
        REQUIRE(it.lo == s.next);  // the CTAs have an item's blocks in their order
        s.next = it.hi;
        if (it.lo == 0) {
          s.first = cta;
          s.nb = it.nb;
          s.pieces = round < cuts.rounds ? 1 : pieces_of(it, walk.at, cuts, cta);
        } else {
          REQUIRE(cta == s.first + s.n);  // where the join looks for it
          ++heads;
        }
        if (it.hi < it.nb) ++tails;
        ++s.n;
        cost += static_cast<int64_t>(it.hi - it.lo) * cost_of(it.rows);
      }
    }
    REQUIRE(heads <= 1 && tails <= 1);  // a slot per CTA each
    REQUIRE(pieces_of_rest >= 1);
    REQUIRE(cost <= cuts.total / cuts.n_pieces + 2 * kCostTwo);
  }
  for (int i = 0; i < shared_items + own_items; ++i) {
    const int nb = i < shared_items ? (ok_prefix ? z.nbp : 0)
                                    : own[(i - shared_items) / z.groups_s % z.B];
    REQUIRE(seen[i].next == nb && seen[i].n == seen[i].pieces);
    REQUIRE(nb == 0 || (seen[i].nb == nb && seen[i].first >= 0 &&
                        seen[i].first + seen[i].n <= kMaxCtas));
  }
  return 0;
}

}  // namespace

// 0, or the line of the check that failed. out: form; rounds and pieces of the few-row
// kernel's line, of the tile kernel's.
extern "C" int check_call(int B, int H_kv, int GL, int d, int prefix_len, int sms, const int* lens,
                          int ok_prefix, int* out) {
  const Form form = form_of(B, GL, prefix_len > 0);
  sms = ctas_of(sms);
  for (int i = 0; i < 5; ++i) out[i] = 0;
  out[0] = form;
  if (form == kFew || form == kMixed) {
    const Sizes z = sizes_of(B, H_kv, GL, d, prefix_len, sms, true, form);
    if (const int at = check_line(z, few_block(d), few_block(d), lens, ok_prefix, false, out + 1)) return at;
  }
  if (form != kFew) {
    const Sizes z = sizes_of(B, H_kv, GL, d, prefix_len, sms, false, form);
    const int64_t items = static_cast<int64_t>(H_kv) *
                          ((z.shared ? z.groups_p : 0) +
                           (z.own ? static_cast<int64_t>(B) * z.groups_s : 0));
    if (const int at = check_line(z, kBK, few_block(d), lens, ok_prefix, items > sms, out + 3)) return at;
  }
  REQUIRE(out[2] + out[4] <= (form == kMixed ? sms : 2 * sms));
  return 0;
}
