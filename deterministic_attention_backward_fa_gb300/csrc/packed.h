// Packed, grouped-head attention and the paged cache: what the host side
// (packed_api.cpp, packed_plan.cpp) and the kernels (packed_fwd.cu,
// packed_bwd.cu, paged.cu) share; api.cpp reads the status word.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace dash {

#ifdef __CUDACC__
template <class T>
struct SameType {
  using type = T;
};
// Launches a kernel and returns the launch's own status.  (What cudaGetLastError
// returns behind <<<>>> may be the error of an earlier call, of a launch that
// went through.)
template <class... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   cudaLaunchAttribute *attr, const typename SameType<P>::type &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = attr ? 1 : 0;
  void *ptrs[] = {const_cast<void *>(static_cast<const void *>(&args))...};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), ptrs);
}
// The kernel may be set up while the one before it runs; it waits for that one's end itself.
inline cudaLaunchAttribute overlap_attr() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
#endif

constexpr int kPackedTile = 128;  // rows of a Q or KV tile; a sequence's tiles start at its first row

// One unit of the packed forward: up to two 128-row Q tiles that read the same
// K/V head over the same sequence (two heads of a group on one tile, or two
// tiles of one head).
struct PackedFwdItem {
  int row0[2];   // first packed row of the tile
  int rows[2];   // valid rows (1..128)
  int nkv[2];    // KV tiles the tile attends; 0: no second tile
  int head[2];   // Q head
  int q0[2];     // position of the first row in its sequence
  int kv_row0;   // packed row of the sequence's first key
  int kv_len;    // keys of the sequence
  int kv_head;
  int pad[3];
};
static_assert(sizeof(PackedFwdItem) == 64, "items are read as four 16-byte words");

struct PackedFwdParams {
  const PackedFwdItem *items;
  const int *cta_off;      // gridDim.x + 1
  __nv_bfloat16 *o;        // row r of head h at o + r * o_row + h * o_head
  long long o_row, o_head;
  float *lse;              // [Hq][lse_head]
  long long lse_head;
  int *status;
  float scale_log2;
  int causal;
  bool wide;             // every 32 bytes of a row of O start at a multiple of 32
  long long spin_limit_ns;
};

// The packed backward's two kernels (packed_bwd.cu).  dQ: one Q tile of one
// head against its KV tiles.
struct PackedDqItem {
  int row0;      // first packed row of the Q tile
  int rows;      // valid rows
  int nkv;       // KV tiles it attends
  int head;      // Q head
  int q0;        // position of its first row in the sequence
  int kv_row0;   // packed row of the sequence's first key
  int kv_len;    // keys of the sequence
  int tile;      // number of the Q tile over all sequences
};
// dK and dV: one KV tile of one K/V head against the Q tiles of its group, or
// the part t0 <= t < t1 of them: its Q tiles q_first .. n - 1 (q_first: the KV
// tile itself, or 0 without the causal mask) of the group's first head, of the
// second head, and so on.
struct PackedDkvItem {
  int row0;      // first packed row of the KV tile
  int rows;      // valid rows
  int kv;        // number of the tile in its sequence
  int head;      // K/V head
  int n;         // tiles of the sequence
  int seq_row0;  // the sequence's first packed row
  int seq_len;
  int tile0;     // number of the sequence's first tile over all sequences
  int t0, t1;    // the part
  int slot;      // -1: the item writes dK and dV; else its sums go to this place of `parts`
  int pad;
};
// A KV tile whose dK and dV were summed in parts.
struct PackedSum {
  int row0, rows, head;
  int slot, n;   // its parts, in their order
  int pad[3];
};
static_assert(sizeof(PackedDqItem) == 32 && sizeof(PackedDkvItem) == 48 && sizeof(PackedSum) == 32,
              "items are read as 16-byte words");

struct PackedBwdParams {
  const PackedDqItem *dq_items;
  const int *dq_off;       // CTA count + 1
  const PackedDkvItem *dkv_items;
  const int *dkv_off;
  const __nv_bfloat16 *o, *dout;
  const float *lse;        // [Hq][lse_head]
  long long o_row, o_head, do_row, do_head, lse_head;
  float *stats;            // [Hq][n_tiles][2][128]: -LSE log2(e) (-inf behind the sequence), -rowsum(dO O)
  const PackedSum *sums;
  int n_sums;
  float *parts;            // [slots][2][128][D]: dV and dK (not yet scaled) of a part
  __nv_bfloat16 *dq, *dk, *dv;
  long long dq_row, dq_head, dk_row, dk_head, dv_row, dv_head;
  int n_tiles, group, causal;
  bool wide_in, wide_dq, wide_dkv;  // as above, of o and dout, dq, and dk, dv and parts
  float scale, scale_log2;
  int *status;
  long long spin_limit_ns;
};
// The kernels, dQ first: it writes the stats that the other reads; then the sums of parts, if any.
cudaError_t launch_packed_bwd(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const CUtensorMap &dout, const PackedBwdParams &p, int dq_ctas, int dkv_ctas,
                              cudaStream_t stream);
cudaError_t prepare_packed_bwd(int D);

cudaError_t launch_packed_fwd(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const PackedFwdParams &p, int num_ctas, cudaStream_t stream);
// Raises the shared-memory limit of the packed kernels and loads them, so that a later call can be captured.
cudaError_t prepare_packed_fwd(int D);


// Address of the current device's status word of the packed and paged kernels.
cudaError_t ops_status_address(int **p);
bool ops_status_used();  // whether any call has asked for it

// ------------------------------------------------------------ paged cache
// Element strides of a cache tensor [pages][tokens][heads][D].
struct CacheStrides {
  long long page, token, head;
};

struct DecodeParams {
  const __nv_bfloat16 *q, *k, *v;
  const int *table, *lengths;
  __nv_bfloat16 *o;
  float *lse;                 // [B][Hq] or null
  float *part_o;              // [B][Hq][max_splits][D], each split's own softmax average
  float2 *part_ml;            // [B][Hq][max_splits] {maximum (scaled, log2), sum}
  long long q_batch, q_head, o_batch, o_head, table_row;
  CacheStrides ks, vs;
  int B, Hq, Hkv, group, n_pages, page_size, max_pages, max_splits;
  int hblocks;                // blocks of 16 Q heads in a group
  float scale_log2;
  int *status;
};
// Tokens a split covers, from the sequence's own length alone.
// Long ones get longer splits (a split's partial result costs as much as eight
// cached tokens to write and read) but up to 64 of them, so that one sequence
// on few heads still spreads.
__host__ __device__ inline int decode_chunk(int len) {
  int c = 256;
  while ((long long)c * 64 < len || (c < 1024 && c * 16 < len)) c *= 2;
  return c;
}
__host__ __device__ inline int decode_splits(int len) {
  const int c = decode_chunk(len);
  return (int)(((long long)len + c - 1) / c);
}
// The most splits that a sequence of up to `cap` tokens can have: a length from
// which splits get longer has more of them than the ones just above it, and
// those lengths are powers of two.
inline int decode_max_splits(int cap) {
  int most = decode_splits(cap);
  for (long long len = 256; len <= cap; len *= 2) {
    const int n = decode_splits((int)len);
    if (n > most) most = n;
  }
  return most;
}
// Whether the splits of a sequence are joined in a cluster (at most 8 CTAs)
// rather than by a second kernel: small calls, whose CTAs all run at once, since
// a cluster waits for 8 free places and holds them to its end.  One sequence of
// 700 to 2000 tokens (16 heads on 4, D = 128) 7.6 us against 8.5 to 9.0 and a
// launch less; 4 of 2000 on 16 K/V heads the same, 8 of them 37.3 against 33.3.
// Clusters of 16 lose (8000 tokens on 16 K/V heads 22.6 against 13.7).
constexpr int kMaxCluster = 8;
inline bool decode_clustered(int B, int Hq, int max_splits) {
  return max_splits > 1 && max_splits <= kMaxCluster && (long long)B * Hq * max_splits <= 512;
}
cudaError_t prepare_decode();  // loads the decode kernels on the current device and raises their shared-memory limit
cudaError_t launch_decode(int D, const DecodeParams &p, int num_sms, cudaStream_t stream);

struct CacheWriteParams {
  const __nv_bfloat16 *k, *v;
  long long k_row, k_head, v_row, v_head;
  __nv_bfloat16 *kp, *vp;
  CacheStrides ks, vs;
  const int *table, *starts, *cu;
  long long table_row;
  int n_tokens, B, heads, D, n_pages, page_size, max_pages;
  int *status;
};
cudaError_t launch_cache_write(const CacheWriteParams &p, int num_sms, cudaStream_t stream);

constexpr int kCopyPairs = 3500;  // pairs in one launch's arguments (at most 32764 bytes)
struct CacheCopyParams {
  __nv_bfloat16 *kp, *vp;
  CacheStrides ks, vs;
  int page_size, heads, D;
};
// pairs: n x {source page, destination page}, on the host.
cudaError_t launch_cache_copy(const CacheCopyParams &p, const int2 *pairs, int n, cudaStream_t stream);

}  // namespace dash
