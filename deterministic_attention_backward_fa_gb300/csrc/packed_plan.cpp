// Host tables of a packed, grouped-head attention problem.
#include "packed_plan.h"

#include <algorithm>
#include <climits>
#include <functional>
#include <numeric>
#include <queue>
#include <utility>

namespace dash {

namespace {

// Cost of an item beside its tiles (its first loads and its last products), in
// tiles: an item's first score and last product have nothing to run under.
constexpr long long kItemCost = 2;
// Keys of one K/V head, both tensors, 128 wide, that fill half of the L2.
constexpr long long kL2Rows = 64LL * 1024 * 1024 / (2 * 128 * 2);

int tiles_of(int len) { return (int)((len + (long long)kPackedTile - 1) / kPackedTile); }

// Sequences by decreasing length, ties in their own order.
std::vector<int> by_length(const PackedTables &t) {
  std::vector<int> order(t.seqs.size());
  std::iota(order.begin(), order.end(), 0);
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return t.seqs[a].y > t.seqs[b].y; });
  return order;
}

// Calls f(sequence, first tile, tiles, first K/V head, end) for every batch of heads.
template <class F>
void for_batches(const PackedTables &t, int Hkv, F f) {
  std::vector<int> tile0(t.seqs.size() + 1, 0);
  for (size_t s = 0; s < t.seqs.size(); ++s) tile0[s + 1] = tile0[s] + tiles_of(t.seqs[s].y);
  for (int s : by_length(t)) {
    if (t.seqs[s].y == 0) break;
    const int batch = (int)std::max<long long>(1, std::min<long long>(Hkv, kL2Rows / t.seqs[s].y));
    for (int h = 0; h < Hkv; h += batch) f(s, tile0[s], tiles_of(t.seqs[s].y), h, std::min(Hkv, h + batch));
  }
}

// Deals the items, in their order, to the CTA with the least work (ties to the
// lowest) and writes them grouped by CTA.  Returns the work of the last CTA to end.
template <class Item, class Cost>
long long deal(const std::vector<Item> &items, int P, Cost cost, std::vector<Item> *out, std::vector<int32_t> *off) {
  using Slot = std::pair<long long, int>;  // {work, CTA}
  P = (int)std::max<long long>(1, std::min<long long>(P, (long long)items.size()));
  std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> heap;
  for (int c = 0; c < P; ++c) heap.push({0, c});
  std::vector<std::vector<int>> lists(P);
  for (size_t i = 0; i < items.size(); ++i) {
    Slot s = heap.top();
    heap.pop();
    lists[s.second].push_back((int)i);
    s.first += cost(items[i]) + kItemCost;
    heap.push(s);
  }
  out->clear();
  out->reserve(items.size());
  off->assign(1, 0);
  for (int c = 0; c < P; ++c) {
    for (int i : lists[c]) out->push_back(items[i]);
    off->push_back((int32_t)out->size());
  }
  long long most = 0;
  for (; !heap.empty(); heap.pop()) most = heap.top().first;
  return most;
}

}  // namespace

std::string packed_sequences(const int32_t *lengths, int n_seqs, PackedTables *out) {
  long long row = 0;
  for (int s = 0; s < n_seqs; ++s) {
    if (lengths[s] < 0) return "length " + std::to_string(s) + " is negative";
    row += lengths[s];
    out->n_tiles += tiles_of(lengths[s]);
  }
  if (row > INT32_MAX - kPackedTile) return "more than 2^31 packed rows";
  out->rows = row;
  out->seqs.resize(n_seqs);
  row = 0;
  for (int s = 0; s < n_seqs; ++s) {
    out->seqs[s] = make_int2((int)row, lengths[s]);
    row += lengths[s];
  }
  return "";
}

void packed_forward(int Hq, int Hkv, bool causal, int P, PackedTables *t) {
  const int group = Hq / Hkv;
  std::vector<PackedFwdItem> items;
  for_batches(*t, Hkv, [&](int seq, int, int n, int h_begin, int h_end) {
    const int2 sq = t->seqs[seq];
    auto tile = [&](PackedFwdItem &it, int half, int qt, int head) {
      it.row0[half] = sq.x + qt * kPackedTile;
      it.rows[half] = std::min(kPackedTile, sq.y - qt * kPackedTile);
      it.nkv[half] = causal ? qt + 1 : n;
      it.head[half] = head;
      it.q0[half] = qt * kPackedTile;
    };
    for (int qt = n - 1; qt >= 0; --qt)
      for (int hk = h_begin; hk < h_end; ++hk) {
        PackedFwdItem base = {};
        base.kv_row0 = sq.x;
        base.kv_len = sq.y;
        base.kv_head = hk;
        const int h0 = hk * group;
        for (int h = 0; h + 1 < group; h += 2) {
          PackedFwdItem it = base;
          tile(it, 0, qt, h0 + h);
          tile(it, 1, qt, h0 + h + 1);
          items.push_back(it);
        }
        if ((group & 1) && (n - 1 - qt) % 2 == 0) {  // the odd head's tiles go in pairs
          PackedFwdItem it = base;
          tile(it, 0, qt, h0 + group - 1);
          if (qt > 0) tile(it, 1, qt - 1, h0 + group - 1);
          items.push_back(it);
        }
      }
  });
  deal(items, P, [](const PackedFwdItem &it) { return (long long)it.nkv[0] + it.nkv[1]; }, &t->fwd, &t->fwd_off);
}

void packed_backward(int Hq, int Hkv, bool causal, int P, PackedTables *t) {
  const int group = Hq / Hkv;
  std::vector<PackedDqItem> dq;
  std::vector<PackedDkvItem> dkv;
  for_batches(*t, Hkv, [&](int seq, int tile0, int n, int h_begin, int h_end) {
    const int2 sq = t->seqs[seq];
    auto rows = [&](int tile) { return std::min(kPackedTile, sq.y - tile * kPackedTile); };
    for (int qt = n - 1; qt >= 0; --qt)
      for (int h = h_begin * group; h < h_end * group; ++h)
        dq.push_back({sq.x + qt * kPackedTile, rows(qt), causal ? qt + 1 : n, h, qt * kPackedTile, sq.x, sq.y,
                      tile0 + qt});
    for (int kv = 0; kv < n; ++kv)
      for (int hk = h_begin; hk < h_end; ++hk)
        dkv.push_back({sq.x + kv * kPackedTile, rows(kv), kv, hk, n, sq.x, sq.y, tile0, 0,
                       group * (causal ? n - kv : n), -1, 0});
  });
  deal(dq, P, [](const PackedDqItem &it) { return (long long)it.nkv; }, &t->dq, &t->dq_off);

  // The dK/dV items are few and large (a KV tile with every Q tile of its
  // group), so balance counts for more than what L2 holds: the longest of all
  // first (a training batch of 16384 tokens 235 us against 246).  Where that
  // still leaves CTAs idle, items longer than `cut` go in parts, whose sums a
  // kernel behind adds up: the cut with the least time, a part costing the bytes
  // that it writes and reads back (about 1 / 40 of a tile pair's time at D = 128,
  // and as much at D = 64, where both are half) and the kernel three tile pairs.
  auto cost = [](const PackedDkvItem &it) { return (long long)it.t1 - it.t0; };
  auto parts_of = [&](long long cut) {
    std::vector<PackedDkvItem> out;
    t->sums.clear();
    t->slots = 0;
    for (const PackedDkvItem &it : dkv) {
      const long long n = (cost(it) + cut - 1) / cut;
      if (n <= 1) {
        out.push_back(it);
        continue;
      }
      t->sums.push_back({it.row0, it.rows, it.head, t->slots, (int)n, {0, 0, 0}});
      for (long long k = 0; k < n; ++k) {
        PackedDkvItem part = it;
        part.t0 = (int)(it.t1 * k / n);
        part.t1 = (int)(it.t1 * (k + 1) / n);
        part.slot = t->slots++;
        out.push_back(part);
      }
    }
    std::stable_sort(out.begin(), out.end(),
                     [&](const PackedDkvItem &a, const PackedDkvItem &b) { return cost(a) > cost(b); });
    return out;
  };
  long long longest = 1, best = -1, best_cut = 0;
  int worse = 0;
  for (const PackedDkvItem &it : dkv) longest = std::max(longest, cost(it));
  for (long long cut = longest; cut >= 4 || cut == longest; cut /= 2) {
    const std::vector<PackedDkvItem> items = parts_of(cut);
    long long time = 40 * deal(items, P, cost, &t->dkv, &t->dkv_off);
    if (t->slots) time += t->slots + 120;
    if (best < 0 || time < best) {
      best = time;
      best_cut = cut;
    } else if (++worse == 2) {
      break;
    }
  }
  deal(parts_of(best_cut), P, cost, &t->dkv, &t->dkv_off);
}

}  // namespace dash
