// C ABI of the 8-bit paged cache (declared in include/dash.h).
#include <new>
#include <vector>

#include "cache8.h"
#include "ops_host.h"

using dash::report;
using namespace dash::host;

namespace {

// The cache of a call; `s`: strides of k_pages, v_pages, k_scales, v_scales, 12 values, or null.
dash_status_t cache8_of(const void *k_pages, const void *v_pages, const void *k_scales, const void *v_scales,
                        int n_pages, int page_size, int Hkv, int D, const int64_t *s, dash::Cache8 *c) {
  dash_status_t st;
  if ((st = check_ptr(k_pages, "k_pages")) || (st = check_ptr(v_pages, "v_pages")) ||
      (st = check_words(k_scales, "k_scales")) || (st = check_words(v_scales, "v_scales")))
    return st;
  const char *names[4] = {"k_pages", "v_pages", "k_scales", "v_scales"};
  dash::CacheStrides *to[4] = {&c->ks, &c->vs, &c->kss, &c->vss};
  for (int i = 0; i < 4; ++i)
    if ((st = cache_strides(s ? s + 3 * i : nullptr, n_pages, page_size, Hkv, i < 2 ? D : 1, names[i], to[i],
                            i < 2 ? 16 : 1)))
      return st;
  c->k = static_cast<uint8_t *>(const_cast<void *>(k_pages));
  c->v = static_cast<uint8_t *>(const_cast<void *>(v_pages));
  c->k_scale = static_cast<float *>(const_cast<void *>(k_scales));
  c->v_scale = static_cast<float *>(const_cast<void *>(v_scales));
  return DASH_OK;
}

// Writing and reading differ in the direction alone.
dash_status_t cache8_rows(bool write, const void *k, const void *v, const void *k_pages, const void *v_pages,
                          const void *k_scales, const void *v_scales, const int32_t *page_table,
                          const int32_t *starts, const int32_t *cu, long long n_tokens, int B, int Hkv, int D,
                          int n_pages, int page_size, int max_pages, const int64_t *strides, dash_stream_t stream) {
  dash_status_t st = check_cache(Hkv, D, n_pages, page_size);
  if (st != DASH_OK) return st;
  if (B < 0 || max_pages < 0 || n_tokens < 0 || n_tokens > INT32_MAX - 65536)
    return report(DASH_ERR_INVALID_ARG, "sizes must be >= 0 and below 2^31");
  if (n_tokens == 0 || (write && B == 0)) return DASH_OK;
  if ((st = check_ptr(k, "k")) || (st = check_ptr(v, "v")) ||
      (st = check_words(page_table, "page_table", max_pages == 0 || B == 0)) ||
      (st = check_words(starts, "starts", B == 0)) || (st = check_words(cu, "cu", B == 0)))
    return st;
  dash::Cache8RowsParams p = {};
  Rows rk, rv;
  if ((st = rows_of(strides, 0, n_tokens, Hkv, D, "k", &rk)) ||
      (st = rows_of(strides, 1, n_tokens, Hkv, D, "v", &rv)) ||
      (st = cache8_of(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D,
                      strides ? strides + 4 : nullptr, &p.c)))
    return st;
  p.table_row = strides ? strides[16] : max_pages;
  if (B > 1 && p.table_row < max_pages) return report(DASH_ERR_INVALID_ARG, "page table rows overlap");
  p.k = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
  p.v = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
  p.k_row = rk.row;
  p.k_head = rk.head;
  p.v_row = rv.row;
  p.v_head = rv.head;
  p.table = page_table;
  p.starts = starts;
  p.cu = cu;
  p.n_tokens = (int)n_tokens;
  p.B = B;
  p.heads = Hkv;
  p.D = D;
  p.n_pages = n_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  const cudaError_t e = (write ? dash::launch_cache8_write : dash::launch_cache8_read)(
      p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, write ? "cache write launch" : "cache read launch");
}

}  // namespace

extern "C" {

dash_status_t dash_cache_write_fp8(const void *k, const void *v, void *k_pages, void *v_pages, float *k_scales,
                                   float *v_scales, const int32_t *page_table, const int32_t *starts,
                                   const int32_t *cu_new, long long n_tokens, int B, int Hkv, int D, int n_pages,
                                   int page_size, int max_pages, const int64_t *strides, dash_stream_t stream) {
  return cache8_rows(true, k, v, k_pages, v_pages, k_scales, v_scales, page_table, starts, cu_new, n_tokens, B, Hkv,
                     D, n_pages, page_size, max_pages, strides, stream);
}

dash_status_t dash_cache_read_fp8(void *k, void *v, const void *k_pages, const void *v_pages, const float *k_scales,
                                  const float *v_scales, const int32_t *page_table, const int32_t *starts,
                                  const int32_t *cu, long long n_tokens, int B, int Hkv, int D, int n_pages,
                                  int page_size, int max_pages, const int64_t *strides, dash_stream_t stream) {
  return cache8_rows(false, k, v, k_pages, v_pages, k_scales, v_scales, page_table, starts, cu, n_tokens, B, Hkv, D,
                     n_pages, page_size, max_pages, strides, stream);
}

dash_status_t dash_cache_copy_fp8(void *k_pages, void *v_pages, float *k_scales, float *v_scales, const int32_t *src,
                                  const int32_t *dst, int n, int Hkv, int D, int n_pages, int page_size,
                                  const int64_t *strides, dash_stream_t stream) try {
  dash_status_t st = check_cache(Hkv, D, n_pages, page_size);
  if (st != DASH_OK) return st;
  if (n < 0) return report(DASH_ERR_INVALID_ARG, "n must be >= 0");
  if (n == 0) return DASH_OK;
  if (!src || !dst) return report(DASH_ERR_INVALID_ARG, "null page list");
  dash::Cache8CopyParams p;
  if ((st = cache8_of(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D, strides, &p.c))) return st;
  std::vector<int2> pairs;
  if ((st = copy_pairs(src, dst, n, n_pages, &pairs)) != DASH_OK) return st;
  p.page_size = page_size;
  p.heads = Hkv;
  p.D = D;
  const cudaError_t e = dash::launch_cache8_copy(p, pairs.data(), n, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "cache copy launch");
} catch (...) {
  return report(DASH_ERR_NO_MEMORY, "cache copy: out of host memory");
}

dash_status_t dash_attn_decode_fp8(const void *q, const void *k_pages, const void *v_pages, const float *k_scales,
                                   const float *v_scales, const int32_t *page_table, const int32_t *lengths, void *o,
                                   float *lse, int B, int Hq, int Hkv, int D, int n_pages, int page_size,
                                   int max_pages, const int64_t *strides, float scale, void *workspace,
                                   long long workspace_bytes, dash_stream_t stream) {
  dash::Decode8Params p = {};
  dash_status_t st = decode_params(q, page_table, lengths, o, lse, B, Hq, Hkv, D, n_pages, page_size, max_pages,
                                   strides, strides ? strides + 16 : nullptr, scale, workspace, workspace_bytes,
                                   dash_decode_workspace(B, Hq, D, page_size, max_pages), 0, 0, &p);
  if (st != DASH_OK || B == 0) return st;
  if ((st = cache8_of(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D,
                      strides ? strides + 4 : nullptr, &p.c)))
    return st;
  p.page = dash::divisor(page_size);
  p.spin_limit_ns = kSpinNs;
  p.whole = page_size % 16 == 0;
  for (const dash::CacheStrides &s : {p.c.ks, p.c.vs, p.c.kss, p.c.vss})
    for (long long x : {s.page, s.token}) p.whole = p.whole && x <= INT32_MAX;
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  const cudaError_t e = dash::launch_decode8(D, p, device.sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "decode launch");
}

}  // extern "C"
