// The 8-bit paged cache: what the entry points (cache8_api.cpp) and the kernels
// (cache8.cu) share.
#pragma once

#include "packed.h"

namespace dash {

// Pages of e4m3 codes [pages][tokens][heads][D] and their rows' fp32 scales
// [pages][tokens][heads]; strides in elements.
struct Cache8 {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  CacheStrides ks, vs, kss, vss;
};

struct Cache8RowsParams {       // write and read
  Cache8 c;
  __nv_bfloat16 *k, *v;         // packed rows; only read by the write
  long long k_row, k_head, v_row, v_head;
  const int *table, *starts, *cu;
  long long table_row;
  int n_tokens, B, heads, D, n_pages, page_size, max_pages;
  int blocks, passes;           // a token's rows are dealt to `blocks` warps, `passes` steps each
  int *status;
};
cudaError_t launch_cache8_write(const Cache8RowsParams &p, cudaStream_t stream);
cudaError_t launch_cache8_read(const Cache8RowsParams &p, cudaStream_t stream);

struct Cache8CopyParams {
  Cache8 c;
  int page_size, heads, D;
};
// pairs: n x {source page, destination page}, on the host.
cudaError_t launch_cache8_copy(const Cache8CopyParams &p, const int2 *pairs, int n, cudaStream_t stream);

// Division of 0 <= n < 2^31 by a divisor d >= 1, as a product:
// n / d = (n + floor(n mul / 2^32)) >> shift, with 2^shift >= d the next power of
// two and mul = floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery).
struct Divisor {
  unsigned mul;
  int shift;
};
inline Divisor divisor(unsigned d) {
  int shift = 0;
  while ((1ull << shift) < d) ++shift;
  return {(unsigned)((((1ull << shift) - d) << 32) / d + 1), shift};
}

struct Decode8Params : DecodeParams {
  Cache8 c;
  Divisor page;  // page_size
  // Steps of 16 tokens lie in one page, and strides fit 32 bits.
  bool whole;
  long long spin_limit_ns;
};
cudaError_t prepare_cache8();
// The form for calls that fill the GPU with groups of up to 8 heads (decode8.cu), but for the join.
cudaError_t prepare_decode8_wide();
cudaError_t launch_decode8_wide(int D, const Decode8Params &p, int num_sms, cudaStream_t stream);
bool encode_pages8_map(CUtensorMap *m, const void *base, int n_pages, int page_size, int heads, int D, long long page,
                       long long token, long long head, int box);  // api.cpp
cudaError_t launch_decode8(int D, const Decode8Params &p, int num_sms, cudaStream_t stream);

}  // namespace dash
