// Host tables of a packed, grouped-head attention problem.
#include "packed_plan.h"

#include <algorithm>
#include <climits>
#include <functional>
#include <numeric>
#include <queue>
#include <utility>

#include "schedule.h"

namespace dash {

namespace {

// Cost of an item of the forward beside its KV tiles (set-up and epilogue), in KV tiles.
constexpr long long kItemCost = 2;

// Keys (of one K/V head, both tensors, 128 wide) that fill half of the L2.
constexpr long long kL2Rows = 64LL * 1024 * 1024 / (2 * 128 * 2);

using Slot = std::pair<long long, int>;  // {load, CTA}: the least loaded, lowest CTA first
using Heap = std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>>;

Heap make_heap(int P) {
  std::vector<Slot> v;
  for (int i = 0; i < P; ++i) v.push_back({0, i});
  return Heap(std::greater<Slot>(), std::move(v));
}

// Sequences by decreasing length, ties in their own order.
std::vector<int> by_length(const PackedTables &t) {
  std::vector<int> order(t.seqs.size());
  std::iota(order.begin(), order.end(), 0);
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return t.seqs[a].y > t.seqs[b].y; });
  return order;
}

}  // namespace

std::string packed_tiles(const int32_t *lengths, int n_seqs, PackedTables *out) {
  long long row = 0, tiles = 0;
  for (int s = 0; s < n_seqs; ++s) {
    if (lengths[s] < 0) return "length " + std::to_string(s) + " is negative";
    row += lengths[s];
    tiles += (lengths[s] + (long long)kPackedTile - 1) / kPackedTile;
  }
  if (row > INT32_MAX - kPackedTile) return "more than 2^31 packed rows";
  out->rows = row;
  out->seqs.resize(n_seqs);
  out->tiles.reserve(tiles);
  row = 0;
  for (int s = 0; s < n_seqs; ++s) {
    const int n = lengths[s];
    out->seqs[s] = make_int2((int)row, n);
    for (int r = 0; r < n; r += kPackedTile)
      out->tiles.push_back(make_int4(r, std::min(kPackedTile, n - r), s, (int)(row + r)));
    row += n;
  }
  return "";
}

void packed_forward(const PackedTables &t, int Hq, int Hkv, bool causal, int P, PackedTables *out) {
  const int group = Hq / Hkv;
  std::vector<PackedFwdItem> items;
  auto tile = [&](PackedFwdItem &it, int half, int seq, int qt, int head) {
    const int2 sq = t.seqs[seq];
    const int n = (sq.y + kPackedTile - 1) / kPackedTile;
    it.row0[half] = sq.x + qt * kPackedTile;
    it.rows[half] = std::min(kPackedTile, sq.y - qt * kPackedTile);
    it.nkv[half] = causal ? qt + 1 : n;
    it.head[half] = head;
    it.q0[half] = qt * kPackedTile;
  };
  for (int seq : by_length(t)) {
    const int2 sq = t.seqs[seq];
    const int n = (sq.y + kPackedTile - 1) / kPackedTile;
    // K/V heads side by side whose keys and values stay in L2 together, all their
    // items the longest first
    const int batch = (int)std::max<long long>(1, std::min<long long>(Hkv, kL2Rows / std::max(1, sq.y)));
    for (int b0 = 0; b0 < Hkv; b0 += batch)
      for (int qt = n - 1; qt >= 0; --qt)
        for (int hk = b0; hk < std::min(Hkv, b0 + batch); ++hk) {
          PackedFwdItem base = {};
          base.kv_row0 = sq.x;
          base.kv_len = sq.y;
          base.kv_head = hk;
          const int h0 = hk * group;
          for (int h = 0; h + 1 < group; h += 2) {
            PackedFwdItem it = base;
            tile(it, 0, seq, qt, h0 + h);
            tile(it, 1, seq, qt, h0 + h + 1);
            items.push_back(it);
          }
          if ((group & 1) && (n - 1 - qt) % 2 == 0) {  // the odd head's tiles go in pairs
            PackedFwdItem it = base;
            tile(it, 0, seq, qt, h0 + group - 1);
            if (qt > 0) tile(it, 1, seq, qt - 1, h0 + group - 1);
            items.push_back(it);
          }
        }
  }
  P = (int)std::max<long long>(1, std::min<long long>(P, (long long)items.size()));
  Heap heap = make_heap(P);
  std::vector<std::vector<int>> lists(P);
  for (size_t i = 0; i < items.size(); ++i) {
    Slot s = heap.top();
    heap.pop();
    lists[s.second].push_back((int)i);
    s.first += items[i].nkv[0] + items[i].nkv[1] + kItemCost;
    heap.push(s);
  }
  out->items.clear();
  out->items.reserve(items.size());
  out->fwd_off.assign(1, 0);
  for (int c = 0; c < P; ++c) {
    for (int i : lists[c]) out->items.push_back(items[i]);
    out->fwd_off.push_back((int32_t)out->items.size());
  }
}

std::string packed_backward(const PackedTables &t, int Hq, int Hkv, bool causal, int P, PackedTables *out) {
  const int group = Hq / Hkv;
  const long long n_tiles = (long long)t.tiles.size();
  long long n_tasks = 0, n_chains = 0;
  for (const int2 &sq : t.seqs) {
    const long long n = (sq.y + kPackedTile - 1) / kPackedTile;
    n_tasks += (causal ? n * (n + 1) / 2 : n * n) * Hq;
    n_chains += n * Hkv;
    if (n > kRankMask) return "a sequence has too many tiles for the task words";
  }
  if (n_tasks > INT32_MAX / 4 || n_tiles * Hq * kSemStride > INT32_MAX)
    return std::to_string(n_tasks) + " tasks: beyond the 32-bit task tables";
  P = (int)std::max<long long>(1, std::min<long long>(P, n_chains));
  struct Chain {
    int hk, kv, seq_tile0, n;  // K/V head, KV tile inside the sequence, the sequence's first tile, its tiles
  };
  Heap heap = make_heap(P);
  std::vector<std::vector<Chain>> lists(P);
  std::vector<int> tile0(t.seqs.size() + 1, 0);
  for (size_t s = 0; s < t.seqs.size(); ++s) tile0[s + 1] = tile0[s] + (t.seqs[s].y + kPackedTile - 1) / kPackedTile;
  for (int seq : by_length(t)) {
    const int n = tile0[seq + 1] - tile0[seq];
    for (int hk = 0; hk < Hkv; ++hk)
      for (int kv = 0; kv < n; ++kv) {  // causal: the longest chain of the head first
        Slot s = heap.top();
        heap.pop();
        lists[s.second].push_back({hk, kv, tile0[seq], n});
        s.first += (long long)group * (causal ? n - kv : n);
        heap.push(s);
      }
  }
  out->tasks.resize((size_t)n_tasks * 4);
  out->bwd_off.assign(1, 0);
  int32_t *w = out->tasks.data();
  int longest = 0;
  for (int c = 0; c < P; ++c) {
    for (const Chain &ch : lists[c]) {
      const int len = causal ? ch.n - ch.kv : ch.n;
      for (int h = 0; h < group; ++h)
        for (int k = 0; k < len; ++k) {
          const int q = causal ? ch.kv + k : (ch.kv + k) % ch.n;
          int32_t word = 0;
          if (h == 0 && k == 0) word |= kTaskFirst;
          if (h == group - 1 && k == len - 1) word |= kTaskLast;
          w[0] = ch.hk * group + h;
          w[1] = ch.seq_tile0 + ch.kv;
          w[2] = ch.seq_tile0 + q;
          w[3] = word;
          w += 4;
        }
    }
    out->bwd_off.push_back((int32_t)((w - out->tasks.data()) / 4));
    longest = std::max(longest, out->bwd_off[c + 1] - out->bwd_off[c]);
  }
  // Ranks in the order of the steps: task i of every CTA before task i + 1 of any.
  std::vector<int32_t> next((size_t)n_tiles * Hq, 0);
  for (int i = 0; i < longest; ++i)
    for (int c = 0; c < P; ++c) {
      if (i >= out->bwd_off[c + 1] - out->bwd_off[c]) continue;
      int32_t *k = out->tasks.data() + 4 * (size_t)(out->bwd_off[c] + i);
      k[3] |= next[(size_t)k[0] * n_tiles + k[2]]++;
    }
  return "";
}

}  // namespace dash
