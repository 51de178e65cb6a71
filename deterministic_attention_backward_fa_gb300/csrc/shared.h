// Decode attention of a batch whose sequences begin with the same tokens: what
// the entry point (ops_api.cpp) and the kernel (shared.cu) share.
#pragma once

#include "packed.h"

namespace dash {

struct SharedParams : DecodeParams {  // first: the prefix; parts_before: its splits
  int prefix_tiles;      // KV tiles of 128 tokens
  int tiles_per_split;
  long long spin_limit_ns;
};

// How the prefix is cut: `splits` runs of `tiles` KV tiles for each K/V head and
// 256 rows (sequence, Q head of the group), so that one wave of CTAs covers all;
// a rule on the sizes alone, whatever the GPU, as the sums go by it.
struct PrefixCut {
  int splits, tiles;
};
constexpr int kPrefixCtas = 152, kMaxPrefixSplits = 64;  // a join holds 128 parts: 64 before, 64 of the tail
inline PrefixCut prefix_cut(int B, int Hq, int Hkv, int prefix) {
  const long long rows = (long long)B * (Hq / Hkv), n = ((long long)prefix + kPackedTile - 1) / kPackedTile;
  const long long base = Hkv * ((rows + 2 * kPackedTile - 1) / (2 * kPackedTile));
  long long splits = kPrefixCtas / base;
  splits = splits < 1 ? 1 : splits > kMaxPrefixSplits ? kMaxPrefixSplits : splits;
  if (splits > n) splits = n;
  const long long tiles = (n + splits - 1) / splits;
  return {(int)((n + tiles - 1) / tiles), (int)tiles};
}

// Whether the prefix is left to dash_decode_kernel, for every sequence by itself:
// where all its splits run at once and are short, what re-reads of the prefix cost
// (they hit L2) is less than two more launches.  4 sequences of 1501 tokens and
// some, 16 heads on 4: 8.1 us against 9.9; 12 of 512 on 8 K/V heads 10.2 and 10.6;
// beyond, 16 of 512 14.7 and 10.7, and one of 4096 in longer splits 11.7 and 11.7.
// It goes by the table's room, as a captured call has to: the 4 sequences with a
// table of more than 4096 tokens take 10.6.
inline bool prefix_with_tails(int B, int Hq, int Hkv, int cap) {
  return decode_chunk(cap) == kMinChunk &&
         (long long)B * Hkv * ((Hq / Hkv + 15) / 16) * decode_max_splits(cap) <= 2 * kPrefixCtas;
}

cudaError_t prepare_shared();
// The prefix, the tails behind it, and their join.
cudaError_t launch_decode_shared(int D, const SharedParams &p, int num_sms, cudaStream_t stream);

}  // namespace dash
