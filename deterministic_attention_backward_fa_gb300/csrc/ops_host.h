// Checks of arguments and device look-ups that the entry points of the packed,
// paged and serving operators share (packed_api.cpp, ops_api.cpp).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <vector>

#include "dash.h"
#include "packed.h"

namespace dash {

dash_status_t report(dash_status_t code, const char *fmt, ...);  // api.cpp

namespace host {

constexpr long long kSpinNs = 2000000000LL;  // 2 s bound on every device wait
constexpr float kLog2e = 1.4426950408889634f;

// A failed call's error stays with the thread until it is taken: left there, a
// later call's check of its launch would find it.
inline dash_status_t cuda_error(cudaError_t e, const char *what) {
  cudaGetLastError();
  return report(DASH_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline dash_status_t check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return report(DASH_ERR_INVALID_ARG, "scale must be finite and > 0");
  return DASH_OK;
}

inline dash_status_t check_ptr(const void *p, const char *name) {
  if (!p) return report(DASH_ERR_INVALID_ARG, "%s is a null pointer", name);
  if (reinterpret_cast<uintptr_t>(p) & 15u) return report(DASH_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return DASH_OK;
}

// Whether every 32-byte piece of a row (of D elements) starts at a multiple of 32.
inline bool wide(const void *p, long long row, long long head) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(row * 2) | (uintptr_t)(head * 2)) & 31u) == 0;
}

// 32-bit values; `optional` ones may be null.
inline dash_status_t check_words(const void *p, const char *name, bool optional = false) {
  if (!p && !optional) return report(DASH_ERR_INVALID_ARG, "%s is a null pointer", name);
  if (reinterpret_cast<uintptr_t>(p) & 3u) return report(DASH_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return DASH_OK;
}

// Tokens of a page table row: the end of the last split and the loads ahead of
// it are counted in 32 bits.
constexpr long long kMaxCached = INT32_MAX - (1 << 26);

// Strides of a [rows][heads][D] tensor, in elements.
struct Rows {
  long long row, head;
};

// Takes strides {row, head} (null: contiguous) and checks that 16-byte vectors
// are aligned and that no two rows share elements.  A stride along an extent of
// one is never used, and set to one that a tensor map takes.
inline dash_status_t rows_of(const int64_t *s, int i, long long rows, int heads, int D, const char *name, Rows *out) {
  Rows r{s ? (long long)s[2 * i] : (long long)heads * D, s ? (long long)s[2 * i + 1] : D};
  if ((rows > 1 && r.row >= (1LL << 38)) || (heads > 1 && r.head >= (1LL << 38)))
    return report(DASH_ERR_UNSUPPORTED, "%s: strides of 2^38 elements and more", name);
  if (rows == 1) r.row = heads > 1 ? std::max<long long>(r.head, D) : D;
  if (heads == 1) r.head = std::max<long long>(r.row, D);
  if (r.row < D || r.head < D || (r.row & 7) || (r.head & 7))
    return report(DASH_ERR_INVALID_ARG, "%s: strides (%lld, %lld) must be multiples of 8 of at least D", name,
                  r.row, r.head);
  if (rows > 1 && heads > 1 && r.row < (heads - 1) * r.head + D && r.head < (rows - 1) * r.row + D)
    return report(DASH_ERR_INVALID_ARG, "%s: its rows overlap", name);
  *out = r;
  return DASH_OK;
}

inline dash_status_t check_heads(int Hq, int Hkv, int D) {
  if (D != 64 && D != 128) return report(DASH_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", D);
  if (Hkv < 1 || Hq < 1 || Hq % Hkv)
    return report(DASH_ERR_INVALID_ARG, "%d Q heads are not a multiple of %d K/V heads", Hq, Hkv);
  if (Hq > 65535) return report(DASH_ERR_UNSUPPORTED, "more than 65535 Q heads");
  return DASH_OK;
}

// What the entry points ask of the current device, looked up once per device:
// the queries and attributes cost more host time than a launch.
struct Device {
  int sms = 0;
  int *status = nullptr;
};
// Of the current device; loads the kernels at its first call.  (packed_api.cpp)
dash_status_t current_device(int *dev, Device *out);

inline dash_status_t cache_strides(const int64_t *s, int n_pages, int page_size, int heads, int D, const char *name,
                                   CacheStrides *out, int step = 8) {
  CacheStrides c{(long long)page_size * heads * D, (long long)heads * D, D};
  if (s) c = {(long long)s[0], (long long)s[1], (long long)s[2]};
  if (n_pages == 1) c.page = 0;
  if (page_size == 1) c.token = 0;
  if (heads == 1) c.head = 0;
  const long long ext[3] = {n_pages, page_size, heads}, st[3] = {c.page, c.token, c.head};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && (st[i] < D || st[i] % step))
      return report(DASH_ERR_INVALID_ARG, "%s: strides (%lld, %lld, %lld) must be multiples of %d of at least %d",
                    name, c.page, c.token, c.head, step, D);
  // walked from the innermost extent outwards, no two rows may share elements
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return st[a] < st[b]; });
  long long span = D;
  for (int i : order) {
    if (ext[i] <= 1) continue;
    if (st[i] < span) return report(DASH_ERR_INVALID_ARG, "%s: its rows overlap", name);
    if (st[i] > (1LL << 60) / ext[i]) return report(DASH_ERR_UNSUPPORTED, "%s: strides too large", name);
    span = (ext[i] - 1) * st[i] + span;
  }
  *out = c;
  return DASH_OK;
}

inline dash_status_t check_cache(int Hkv, int D, int n_pages, int page_size) {
  if (n_pages < 1 || page_size < 1) return report(DASH_ERR_INVALID_ARG, "the cache needs pages and tokens in a page");
  if (Hkv < 1) return report(DASH_ERR_INVALID_ARG, "the cache needs heads");
  if (D != 64 && D != 128) return report(DASH_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", D);
  // a page's 16-byte vectors, with the strides of the loops over them, are counted in 32 bits
  if ((long long)page_size * Hkv * (D / 8) > INT32_MAX / 2) return report(DASH_ERR_UNSUPPORTED, "pages too large");
  return DASH_OK;
}

// The pairs of a copy inside a cache, unless their result would depend on an order.
inline dash_status_t copy_pairs(const int32_t *src, const int32_t *dst, int n, int n_pages, std::vector<int2> *out) {
  std::vector<bool> to(n_pages);
  for (int i = 0; i < n; ++i) {
    if (dst[i] < 0 || dst[i] >= n_pages)
      return report(DASH_ERR_INVALID_ARG, "destination page %d outside the cache's %d pages", dst[i], n_pages);
    if (to[dst[i]]) return report(DASH_ERR_INVALID_ARG, "destination page %d is named twice", dst[i]);
    to[dst[i]] = true;
  }
  out->resize(n);
  for (int i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= n_pages)
      return report(DASH_ERR_INVALID_ARG, "source page %d outside the cache's %d pages", src[i], n_pages);
    if (to[src[i]])
      return report(DASH_ERR_INVALID_ARG, "page %d is a source and a destination of one call", src[i]);
    (*out)[i] = make_int2(src[i], dst[i]);
  }
  return DASH_OK;
}

// All of a decode's parameters but those of the cache itself.  strides: q
// {batch, head}, o {batch, head}, then others; table_row: the page table's;
// `need`: bytes of workspace; the first `first` tokens leave `parts_before` parts.
inline dash_status_t decode_params(const void *q, const int32_t *page_table, const int32_t *lengths, void *o,
                                   float *lse, int B, int Hq, int Hkv, int D, int n_pages, int page_size,
                                   int max_pages, const int64_t *strides, const int64_t *table_row, float scale,
                                   void *workspace, long long workspace_bytes, long long need, int first,
                                   int parts_before, DecodeParams *out) {
  dash_status_t st = check_scale(scale);
  if (st != DASH_OK || (st = check_heads(Hq, Hkv, D)) || (st = check_cache(Hkv, D, n_pages, page_size))) return st;
  if (B < 0 || max_pages < 0) return report(DASH_ERR_INVALID_ARG, "B and max_pages must be >= 0");
  if ((long long)page_size * max_pages > kMaxCached)
    return report(DASH_ERR_UNSUPPORTED, "a page table row covers more than %lld tokens (2^31 less 2^26)", kMaxCached);
  if (B > 65535) return report(DASH_ERR_UNSUPPORTED, "more than 65535 sequences");
  if (B == 0) return DASH_OK;
  if ((st = check_ptr(q, "q")) || (st = check_ptr(o, "o"))) return st;
  if ((st = check_words(page_table, "page_table", max_pages == 0)) || (st = check_words(lengths, "lengths")) ||
      (st = check_words(lse, "lse", true)))
    return st;
  Rows rq, ro;
  if ((st = rows_of(strides, 0, B, Hq, D, "q", &rq)) || (st = rows_of(strides, 1, B, Hq, D, "o", &ro))) return st;
  DecodeParams &p = *out;
  p.table_row = table_row ? *table_row : max_pages;
  if (B > 1 && p.table_row < max_pages) return report(DASH_ERR_INVALID_ARG, "page table rows overlap");
  p.max_splits = std::max(1, decode_max_splits(page_size * max_pages - first));
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need))
    return report(DASH_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", need);
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k = p.v = nullptr;
  p.table = page_table;
  p.lengths = lengths;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)B * Hq * (parts_before + p.max_splits) * D);
  p.q_batch = rq.row;
  p.q_head = rq.head;
  p.o_batch = ro.row;
  p.o_head = ro.head;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.group = Hq / Hkv;
  p.n_pages = n_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.hblocks = (p.group + 15) / 16;
  p.first = first;
  p.shared = 0;
  p.parts_before = parts_before;
  p.least_chunk = kMinChunk;
  p.scale_log2 = scale * kLog2e;
  return DASH_OK;
}

// A decode's bf16 cache; strides: q, o, then k_pages and v_pages.
inline dash_status_t decode_cache(const void *k_pages, const void *v_pages, int Hkv, int D, int n_pages,
                                  int page_size, const int64_t *strides, DecodeParams *p) {
  dash_status_t st;
  if ((st = check_ptr(k_pages, "k_pages")) || (st = check_ptr(v_pages, "v_pages")) ||
      (st = cache_strides(strides ? strides + 4 : nullptr, n_pages, page_size, Hkv, D, "k_pages", &p->ks)) ||
      (st = cache_strides(strides ? strides + 7 : nullptr, n_pages, page_size, Hkv, D, "v_pages", &p->vs)))
    return st;
  p->k = static_cast<const __nv_bfloat16 *>(k_pages);
  p->v = static_cast<const __nv_bfloat16 *>(v_pages);
  return DASH_OK;
}

}  // namespace host
}  // namespace dash
