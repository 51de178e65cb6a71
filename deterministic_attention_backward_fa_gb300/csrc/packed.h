// Packed, grouped-head attention and the paged cache: what the host side
// (packed.cpp) and the kernels (packed_fwd.cu, bwd.cu, packed_bwd.cu,
// paged.cu) share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace dash {

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
  long long spin_limit_ns;
};

// Preprocess of the packed backward: per (Q head, tile) the padded rows' lse2
// and delta, the semaphore's zero, and each sequence's four tensor maps.
struct PackedPreParams {
  const __nv_bfloat16 *o, *dout;
  const float *lse;  // [Hq][lse_head]
  long long o_row, o_head, do_row, do_head, lse_head;
  const int4 *tiles;
  const int2 *seqs;  // {first packed row, length}
  float *lse2, *delta;
  int *sem;
  CUtensorMap *maps;
  const void *base[4];       // Q, K, V, dO
  long long base_row[4];     // their row strides in bytes
  int n_tiles, n_seqs, heads;
};
cudaError_t launch_packed_preprocess(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                     const CUtensorMap &dout, const PackedPreParams &p, cudaStream_t stream);

struct PackedConvertParams {
  const float *accum;        // [Hq][n_tiles][D/4][128][4]
  const int4 *tiles;
  __nv_bfloat16 *dq;
  long long dq_row, dq_head;
  float scale;
  int n_tiles, heads;
};
cudaError_t launch_packed_convert(int D, const PackedConvertParams &p, cudaStream_t stream);

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
__host__ __device__ inline int decode_chunk(int len) {
  int c = 256;
  while ((long long)c * 128 < len) c *= 2;
  return c;
}
__host__ __device__ inline int decode_splits(int len) {
  const int c = decode_chunk(len);
  return (int)(((long long)len + c - 1) / c);
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
