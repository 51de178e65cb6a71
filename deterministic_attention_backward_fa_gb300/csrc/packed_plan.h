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
  long long rows = 0, n_tiles = 0;     // sums over the sequences
  // items grouped by CTA, each with CTA count + 1 offsets
  std::vector<PackedFwdItem> fwd;
  std::vector<PackedDqItem> dq;
  std::vector<PackedDkvItem> dkv;
  std::vector<PackedSum> sums;         // KV tiles whose items are parts
  int slots = 0;                       // parts
  std::vector<int32_t> fwd_off, dq_off, dkv_off;
};

// Lengths and tiles.  Empty string on success, else the reason.
std::string packed_sequences(const int32_t *lengths, int n_seqs, PackedTables *out);

// The items of the forward and of the backward's two kernels on up to P CTAs:
// sequences by decreasing length, inside one the K/V heads in batches whose keys
// and values fit in L2 together, inside a batch the longest items first (dK and
// dV: the longest items of all first), each to the CTA that has the least work
// so far.
void packed_forward(int Hq, int Hkv, bool causal, int P, PackedTables *t);
void packed_backward(int Hq, int Hkv, bool causal, int P, PackedTables *t);

}  // namespace dash
