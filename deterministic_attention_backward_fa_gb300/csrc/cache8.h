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
  int *status;
};
cudaError_t launch_cache8_write(const Cache8RowsParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache8_read(const Cache8RowsParams &p, int num_sms, cudaStream_t stream);

struct Cache8CopyParams {
  Cache8 c;
  int page_size, heads, D;
};
// pairs: n x {source page, destination page}, on the host.
cudaError_t launch_cache8_copy(const Cache8CopyParams &p, const int2 *pairs, int n, cudaStream_t stream);

struct Decode8Params : DecodeParams {
  Cache8 c;
};
cudaError_t prepare_cache8();
cudaError_t launch_decode8(int D, const Decode8Params &p, int num_sms, cudaStream_t stream);

}  // namespace dash
