// Tables of a packed, grouped-head attention problem.  Pure host C++; see
// packed_plan.cpp.
#pragma once

#include <cstdint>
#include <string>
#include <vector>

#include "packed.h"

namespace dash {

struct PackedTables {
  std::vector<int2> seqs;              // {first packed row, length}
  std::vector<int4> tiles;             // {first row inside the sequence, valid rows, sequence, first packed row}
  std::vector<PackedFwdItem> items;    // grouped by CTA
  std::vector<int32_t> fwd_off;        // CTA count + 1
  std::vector<int32_t> tasks;          // backward: {Q head, KV tile, Q tile, rank | flags}, grouped by CTA
  std::vector<int32_t> bwd_off;        // CTA count + 1
  long long rows = 0;                  // sum of the lengths
};

// Lengths and tiles.  Empty string on success, else the reason.
std::string packed_tiles(const int32_t *lengths, int n_seqs, PackedTables *out);

// The forward's items on up to P CTAs: the most work first, each to the CTA
// that has the least so far.
void packed_forward(const PackedTables &t, int Hq, int Hkv, bool causal, int P, PackedTables *out);

// The backward's task table on up to P CTAs.  A chain is one KV tile of one
// K/V head with every Q head of its group; chains go, the longest of a
// sequence first, to the CTA that is free first, each task taking one step.  A
// dQ tile's partials are added in the order of those steps (ties by CTA), so
// the ranks grow along every CTA's list and no cycle of waits can arise.
// Empty string on success, else the reason.
std::string packed_backward(const PackedTables &t, int Hq, int Hkv, bool causal, int P, PackedTables *out);

}  // namespace dash
