// C ABI of the packed attention and the paged cache (declared in include/dash.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "cache8.h"
#include "dash.h"
#include "norm_rope.h"
#include "packed.h"
#include "ops_host.h"
#include "packed_plan.h"
#include "shared.h"

namespace dash {
dash_status_t encode_rows_map(CUtensorMap *m, const void *base, int heads, long long rows, int D,
                              long long row_stride, long long head_stride, int box_rows);
}  // namespace dash

using dash::report;
using namespace dash::host;

// A plan: the tables of one set of lengths on the device it was made on.
struct dash_packed_plan_st {
  long long spin_ns = kSpinNs;
  int device = 0, Hq = 0, Hkv = 0, D = 0, causal = 0, n_seqs = 0;
  long long rows = 0, n_tiles = 0;
  int fwd_ctas = 0, dq_ctas = 0, dkv_ctas = 0;
  bool backward = false;
  void *mem = nullptr;
  const dash::PackedFwdItem *fwd = nullptr;
  const dash::PackedDqItem *dq = nullptr;
  const dash::PackedDkvItem *dkv = nullptr;
  const dash::PackedSum *sums = nullptr;
  int n_sums = 0, slots = 0;
  const int *fwd_off = nullptr, *dq_off = nullptr, *dkv_off = nullptr;
  int *status = nullptr;
};

namespace {

// Workspace of a packed backward: two floats for every row of every tile and
// head, then dV and dK of the KV tiles that are summed in parts.
long long stats_bytes(const dash_packed_plan_st *p) { return p->n_tiles * p->Hq * 2 * dash::kPackedTile * 4; }
long long bwd_bytes(const dash_packed_plan_st *p) {
  return stats_bytes(p) + (long long)p->slots * 2 * dash::kPackedTile * p->D * 4;
}

dash_status_t check_plan(const dash_packed_plan_st *p, long long rows) {
  if (!p) return report(DASH_ERR_INVALID_ARG, "null plan");
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
  if (dev != p->device)
    return report(DASH_ERR_INVALID_ARG, "the plan was made on device %d, the current device is %d", p->device, dev);
  if (rows < p->rows)
    return report(DASH_ERR_INVALID_ARG, "%lld rows are fewer than the plan's %lld", rows, p->rows);
  if (rows > INT32_MAX - dash::kPackedTile) return report(DASH_ERR_UNSUPPORTED, "more than 2^31 packed rows");
  return DASH_OK;
}

std::mutex g_devices_mu;
std::map<int, Device> g_devices;

}  // namespace

dash_status_t dash::host::current_device(int *dev, Device *out) try {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lock(g_devices_mu);
  Device &d = g_devices[*dev];
  if (!d.status) {
    // the first call may come inside a capture, which loading the kernels is no part of
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, *dev)) != cudaSuccess ||
        (e = dash::prepare_decode()) != cudaSuccess || (e = dash::prepare_norm_rope()) != cudaSuccess ||
        (e = dash::prepare_cache8()) != cudaSuccess || (e = dash::prepare_shared()) != cudaSuccess ||
        (e = dash::ops_status_address(&d.status)) != cudaSuccess)
      d.status = nullptr;
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return cuda_error(e, "device set-up");
  }
  *out = d;
  return DASH_OK;
} catch (...) {
  return report(DASH_ERR_NO_MEMORY, "device set-up: out of host memory");
}

extern "C" {

dash_status_t dash_packed_plan_create(const int32_t *lengths, int n_seqs, int Hq, int Hkv, int D, int causal,
                                      int backward, dash_packed_plan_t **plan_out) try {
  if (!plan_out) return report(DASH_ERR_INVALID_ARG, "null plan pointer");
  *plan_out = nullptr;
  if (n_seqs < 0 || (n_seqs > 0 && !lengths)) return report(DASH_ERR_INVALID_ARG, "null lengths");
  dash_status_t st = check_heads(Hq, Hkv, D);
  if (st != DASH_OK) return st;
  dash::PackedTables t;
  std::string why = dash::packed_sequences(lengths, n_seqs, &t);
  if (!why.empty()) return report(DASH_ERR_INVALID_ARG, "%s", why.c_str());
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  std::unique_ptr<dash_packed_plan_st> p(new dash_packed_plan_st());
  p->device = dev;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->D = D;
  p->causal = causal ? 1 : 0;
  p->n_seqs = n_seqs;
  p->rows = t.rows;
  p->n_tiles = t.n_tiles;
  p->backward = backward != 0;
  if (t.rows > 0) {
    if (t.n_tiles * Hq > INT32_MAX / 4)
      return report(DASH_ERR_UNSUPPORTED, "%lld tiles of %d heads: beyond the 32-bit tables", t.n_tiles, Hq);
    dash::packed_forward(Hq, Hkv, causal != 0, device.sms, &t);
    p->fwd_ctas = (int)t.fwd_off.size() - 1;
    if (backward) {
      dash::packed_backward(Hq, Hkv, causal != 0, device.sms, &t);
      p->dq_ctas = (int)t.dq_off.size() - 1;
      p->dkv_ctas = (int)t.dkv_off.size() - 1;
      p->n_sums = (int)t.sums.size();
      p->slots = t.slots;
    }
    cudaError_t e = dash::prepare_packed_fwd(D);
    if (e != cudaSuccess) return cuda_error(e, "packed forward");
    if (backward && (e = dash::prepare_packed_bwd(D)) != cudaSuccess) return cuda_error(e, "packed backward");
    p->status = device.status;
    // one block of device memory, copied once
    std::vector<uint8_t> host;
    auto put = [&](const void *src, size_t bytes) {
      const size_t at = (host.size() + 255) / 256 * 256;
      host.resize(at + bytes);
      if (bytes) std::memcpy(host.data() + at, src, bytes);
      return at;
    };
    auto table = [&](const auto &v) { return put(v.data(), v.size() * sizeof(v[0])); };
    const size_t at[7] = {table(t.fwd), table(t.fwd_off), table(t.dq),  table(t.dq_off),
                          table(t.dkv), table(t.dkv_off), table(t.sums)};
    if ((e = cudaMalloc(&p->mem, host.size())) != cudaSuccess) {
      cudaGetLastError();
      return report(e == cudaErrorMemoryAllocation ? DASH_ERR_NO_MEMORY : DASH_ERR_CUDA, "plan of %zu bytes: %s",
                    host.size(), cudaGetErrorString(e));
    }
    // pageable memory: cudaMemcpy may return with the copy's last step on its way, and the streams that use the
    // plan need not wait for this one
    if ((e = cudaMemcpy(p->mem, host.data(), host.size(), cudaMemcpyHostToDevice)) != cudaSuccess ||
        (e = cudaStreamSynchronize(cudaStreamLegacy)) != cudaSuccess) {
      cudaFree(p->mem);
      return cuda_error(e, "plan tables");
    }
    uint8_t *m = static_cast<uint8_t *>(p->mem);
    p->fwd = reinterpret_cast<const dash::PackedFwdItem *>(m + at[0]);
    p->fwd_off = reinterpret_cast<const int *>(m + at[1]);
    p->dq = reinterpret_cast<const dash::PackedDqItem *>(m + at[2]);
    p->dq_off = reinterpret_cast<const int *>(m + at[3]);
    p->dkv = reinterpret_cast<const dash::PackedDkvItem *>(m + at[4]);
    p->dkv_off = reinterpret_cast<const int *>(m + at[5]);
    p->sums = reinterpret_cast<const dash::PackedSum *>(m + at[6]);
  }
  *plan_out = p.release();
  return DASH_OK;
} catch (const std::bad_alloc &) {
  return report(DASH_ERR_NO_MEMORY, "plan: out of host memory");
} catch (...) {
  return report(DASH_ERR_NO_MEMORY, "plan: the host tables could not be built");
}

void dash_packed_plan_destroy(dash_packed_plan_t *plan) {
  if (!plan) return;
  if (plan->mem) {
    int dev = 0;
    const bool other = cudaGetDevice(&dev) == cudaSuccess && dev != plan->device;
    if (other) cudaSetDevice(plan->device);
    // a plan may be dropped while some thread captures a graph; freeing its memory is no part of that graph
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    cudaFree(plan->mem);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (other) cudaSetDevice(dev);
  }
  delete plan;
}

dash_status_t dash_packed_plan_spin_limit(dash_packed_plan_t *plan, long long ns) {
  if (!plan) return report(DASH_ERR_INVALID_ARG, "null plan");
  if (ns < 0) return report(DASH_ERR_INVALID_ARG, "the spin limit must be >= 0");
  plan->spin_ns = ns ? ns : kSpinNs;
  return DASH_OK;
}

long long dash_packed_bwd_workspace(const dash_packed_plan_t *plan) {
  if (!plan || !plan->backward) return -1;
  return bwd_bytes(plan);
}

dash_status_t dash_build_packed_items(const int32_t *lengths, int n_seqs, int Hq, int Hkv, int causal, int kernel,
                                      int P, int32_t *items_out, int32_t *cta_off_out, int *ctas_out,
                                      long long *n_items_out) try {
  if (n_seqs < 0 || (n_seqs > 0 && !lengths) || P < 1 || kernel < 0 || kernel > 2 || !n_items_out)
    return report(DASH_ERR_INVALID_ARG, "dash_build_packed_items: null pointer or sizes out of range");
  dash_status_t st = check_heads(Hq, Hkv, 64);
  if (st != DASH_OK) return st;
  dash::PackedTables t;
  std::string why = dash::packed_sequences(lengths, n_seqs, &t);
  if (!why.empty()) return report(DASH_ERR_INVALID_ARG, "%s", why.c_str());
  if (t.n_tiles * Hq > INT32_MAX / 4)
    return report(DASH_ERR_UNSUPPORTED, "%lld tiles of %d heads: beyond the 32-bit tables", t.n_tiles, Hq);
  if (kernel == 0)
    dash::packed_forward(Hq, Hkv, causal != 0, P, &t);
  else
    dash::packed_backward(Hq, Hkv, causal != 0, P, &t);
  const std::vector<int32_t> &off = kernel == 0 ? t.fwd_off : kernel == 1 ? t.dq_off : t.dkv_off;
  const void *items = kernel == 0 ? (const void *)t.fwd.data() : kernel == 1 ? (const void *)t.dq.data() : t.dkv.data();
  const size_t size = kernel == 0   ? sizeof(dash::PackedFwdItem)
                      : kernel == 1 ? sizeof(dash::PackedDqItem)
                                    : sizeof(dash::PackedDkvItem);
  *n_items_out = off.back();
  if (ctas_out) *ctas_out = (int)off.size() - 1;
  if (items_out && off.back()) std::memcpy(items_out, items, off.back() * size);
  if (cta_off_out) std::memcpy(cta_off_out, off.data(), off.size() * 4);
  return DASH_OK;
} catch (...) {
  return report(DASH_ERR_NO_MEMORY, "dash_build_packed_items: out of host memory");
}

dash_status_t dash_attn_packed_fwd(const dash_packed_plan_t *plan, const void *q, const void *k, const void *v,
                                   void *o, float *lse, long long rows, const int64_t *strides, float scale,
                                   dash_stream_t stream) {
  dash_status_t st = check_scale(scale);
  if (st != DASH_OK || (st = check_plan(plan, rows)) != DASH_OK) return st;
  if (plan->rows == 0) return DASH_OK;
  if ((st = check_ptr(q, "q")) || (st = check_ptr(k, "k")) || (st = check_ptr(v, "v")) || (st = check_ptr(o, "o")))
    return st;
  if ((st = check_words(lse, "lse")) != DASH_OK) return st;
  const int D = plan->D;
  Rows rq, rk, rv, ro;
  if ((st = rows_of(strides, 0, rows, plan->Hq, D, "q", &rq)) ||
      (st = rows_of(strides, 1, rows, plan->Hkv, D, "k", &rk)) ||
      (st = rows_of(strides, 2, rows, plan->Hkv, D, "v", &rv)) ||
      (st = rows_of(strides, 3, rows, plan->Hq, D, "o", &ro)))
    return st;
  CUtensorMap mq, mk, mv;
  if ((st = dash::encode_rows_map(&mq, q, plan->Hq, rows, D, rq.row, rq.head, dash::kPackedTile)) ||
      (st = dash::encode_rows_map(&mk, k, plan->Hkv, rows, D, rk.row, rk.head, dash::kPackedTile)) ||
      (st = dash::encode_rows_map(&mv, v, plan->Hkv, rows, D, rv.row, rv.head, dash::kPackedTile)))
    return st;
  dash::PackedFwdParams p;
  p.items = plan->fwd;
  p.cta_off = plan->fwd_off;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.o_row = ro.row;
  p.o_head = ro.head;
  p.lse = lse;
  p.lse_head = rows;
  p.status = plan->status;
  p.scale_log2 = scale * kLog2e;
  p.causal = plan->causal;
  p.wide = wide(o, ro.row, ro.head);
  p.spin_limit_ns = plan->spin_ns;
  const cudaError_t e =
      dash::launch_packed_fwd(D, mq, mk, mv, p, plan->fwd_ctas, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "packed forward launch");
}

dash_status_t dash_attn_packed_bwd(const dash_packed_plan_t *plan, const void *q, const void *k, const void *v,
                                   const void *o, const void *dout, const float *lse, void *dq, void *dk, void *dv,
                                   long long rows, const int64_t *strides, float scale, void *workspace,
                                   long long workspace_bytes, dash_stream_t stream) {
  dash_status_t st = check_scale(scale);
  if (st != DASH_OK || (st = check_plan(plan, rows)) != DASH_OK) return st;
  if (!plan->backward) return report(DASH_ERR_INVALID_ARG, "the plan was made without its backward");
  if (plan->rows == 0) return DASH_OK;
  const void *ptrs[8] = {q, k, v, o, dout, dq, dk, dv};
  const char *names[8] = {"q", "k", "v", "o", "dout", "dq", "dk", "dv"};
  const int heads[8] = {plan->Hq, plan->Hkv, plan->Hkv, plan->Hq, plan->Hq, plan->Hq, plan->Hkv, plan->Hkv};
  Rows r[8];
  for (int i = 0; i < 8; ++i)
    if ((st = check_ptr(ptrs[i], names[i])) || (st = rows_of(strides, i, rows, heads[i], plan->D, names[i], &r[i])))
      return st;
  if ((st = check_words(lse, "lse")) != DASH_OK) return st;
  const long long need = bwd_bytes(plan);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need)
    return report(DASH_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", need);
  CUtensorMap m[4];
  const int of[4] = {0, 1, 2, 4};  // Q, K, V, dO
  for (int i = 0; i < 4; ++i) {
    const int x = of[i];
    if ((st = dash::encode_rows_map(&m[i], ptrs[x], heads[x], rows, plan->D, r[x].row, r[x].head,
                                    dash::kPackedTile)) != DASH_OK)
      return st;
  }
  dash::PackedBwdParams p;
  p.dq_items = plan->dq;
  p.dq_off = plan->dq_off;
  p.dkv_items = plan->dkv;
  p.dkv_off = plan->dkv_off;
  p.o = static_cast<const __nv_bfloat16 *>(o);
  p.dout = static_cast<const __nv_bfloat16 *>(dout);
  p.lse = lse;
  p.o_row = r[3].row;
  p.o_head = r[3].head;
  p.do_row = r[4].row;
  p.do_head = r[4].head;
  p.lse_head = rows;
  p.stats = static_cast<float *>(workspace);
  p.parts = p.stats + stats_bytes(plan) / 4;
  p.sums = plan->sums;
  p.n_sums = plan->n_sums;
  p.dq = static_cast<__nv_bfloat16 *>(dq);
  p.dk = static_cast<__nv_bfloat16 *>(dk);
  p.dv = static_cast<__nv_bfloat16 *>(dv);
  p.dq_row = r[5].row;
  p.dq_head = r[5].head;
  p.dk_row = r[6].row;
  p.dk_head = r[6].head;
  p.dv_row = r[7].row;
  p.dv_head = r[7].head;
  p.n_tiles = (int)plan->n_tiles;
  p.group = plan->Hq / plan->Hkv;
  p.causal = plan->causal;
  bool w[8];
  for (int i = 0; i < 8; ++i) w[i] = wide(ptrs[i], r[i].row, r[i].head);
  p.wide_in = w[3] && w[4];
  p.wide_dq = w[5];
  p.wide_dkv = w[6] && w[7] && wide(p.parts, 0, 0);
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.status = plan->status;
  p.spin_limit_ns = plan->spin_ns;
  const cudaError_t e = dash::launch_packed_bwd(plan->D, m[0], m[1], m[2], m[3], p, plan->dq_ctas, plan->dkv_ctas,
                                                reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "packed backward launch");
}

long long dash_decode_workspace(int B, int Hq, int D, int page_size, int max_pages) {
  if (B < 0 || Hq < 1 || (D != 64 && D != 128) || page_size < 1 || max_pages < 0 ||
      (long long)page_size * max_pages > kMaxCached)
    return -1;
  const int splits = dash::decode_max_splits(page_size * max_pages);
  return splits <= 1 || dash::decode_clustered(B, Hq, splits) ? 0 : (long long)B * Hq * splits * (D * 4 + 8) + 256;
}

dash_status_t dash_attn_decode(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                               const int32_t *lengths, void *o, float *lse, int B, int Hq, int Hkv, int D,
                               int n_pages, int page_size, int max_pages, const int64_t *strides, float scale,
                               void *workspace, long long workspace_bytes, dash_stream_t stream) {
  dash::DecodeParams p;
  dash_status_t st = decode_params(q, page_table, lengths, o, lse, B, Hq, Hkv, D, n_pages, page_size, max_pages,
                                   strides, strides ? strides + 10 : nullptr, scale, workspace, workspace_bytes,
                                   dash_decode_workspace(B, Hq, D, page_size, max_pages), 0, 0, &p);
  if (st != DASH_OK || B == 0) return st;
  if ((st = decode_cache(k_pages, v_pages, Hkv, D, n_pages, page_size, strides, &p)) != DASH_OK) return st;
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  const cudaError_t e = dash::launch_decode(D, p, device.sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "decode launch");
}

dash_status_t dash_cache_write(const void *k, const void *v, void *k_pages, void *v_pages,
                               const int32_t *page_table, const int32_t *starts, const int32_t *cu_new,
                               long long n_tokens, int B, int Hkv, int D, int n_pages, int page_size, int max_pages,
                               const int64_t *strides, dash_stream_t stream) {
  dash_status_t st = check_cache(Hkv, D, n_pages, page_size);
  if (st != DASH_OK) return st;
  if (B < 0 || max_pages < 0 || n_tokens < 0 || n_tokens > INT32_MAX - 65536)
    return report(DASH_ERR_INVALID_ARG, "sizes must be >= 0 and below 2^31");
  if (B == 0 || n_tokens == 0) return DASH_OK;
  if ((st = check_ptr(k, "k")) || (st = check_ptr(v, "v")) || (st = check_ptr(k_pages, "k_pages")) ||
      (st = check_ptr(v_pages, "v_pages")))
    return st;
  if ((st = check_words(page_table, "page_table", max_pages == 0)) || (st = check_words(starts, "starts")) ||
      (st = check_words(cu_new, "cu_new")))
    return st;
  Rows rk, rv;
  if ((st = rows_of(strides, 0, n_tokens, Hkv, D, "k", &rk)) || (st = rows_of(strides, 1, n_tokens, Hkv, D, "v", &rv)))
    return st;
  dash::CacheWriteParams p;
  if ((st = cache_strides(strides ? strides + 4 : nullptr, n_pages, page_size, Hkv, D, "k_pages", &p.ks)) ||
      (st = cache_strides(strides ? strides + 7 : nullptr, n_pages, page_size, Hkv, D, "v_pages", &p.vs)))
    return st;
  p.table_row = strides ? strides[10] : max_pages;
  if (B > 1 && p.table_row < max_pages) return report(DASH_ERR_INVALID_ARG, "page table rows overlap");
  p.k = static_cast<const __nv_bfloat16 *>(k);
  p.v = static_cast<const __nv_bfloat16 *>(v);
  p.k_row = rk.row;
  p.k_head = rk.head;
  p.v_row = rv.row;
  p.v_head = rv.head;
  p.kp = static_cast<__nv_bfloat16 *>(k_pages);
  p.vp = static_cast<__nv_bfloat16 *>(v_pages);
  p.table = page_table;
  p.starts = starts;
  p.cu = cu_new;
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
  const cudaError_t e = dash::launch_cache_write(p, device.sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "cache write launch");
}

dash_status_t dash_cache_copy(void *k_pages, void *v_pages, const int32_t *src, const int32_t *dst, int n, int Hkv,
                              int D, int n_pages, int page_size, const int64_t *strides, dash_stream_t stream) try {
  dash_status_t st = check_cache(Hkv, D, n_pages, page_size);
  if (st != DASH_OK) return st;
  if (n < 0) return report(DASH_ERR_INVALID_ARG, "n must be >= 0");
  if (n == 0) return DASH_OK;
  if (!src || !dst) return report(DASH_ERR_INVALID_ARG, "null page list");
  if ((st = check_ptr(k_pages, "k_pages")) || (st = check_ptr(v_pages, "v_pages"))) return st;
  dash::CacheCopyParams p;
  if ((st = cache_strides(strides, n_pages, page_size, Hkv, D, "k_pages", &p.ks)) ||
      (st = cache_strides(strides ? strides + 3 : nullptr, n_pages, page_size, Hkv, D, "v_pages", &p.vs)))
    return st;
  std::vector<int2> pairs;
  if ((st = copy_pairs(src, dst, n, n_pages, &pairs)) != DASH_OK) return st;
  p.kp = static_cast<__nv_bfloat16 *>(k_pages);
  p.vp = static_cast<__nv_bfloat16 *>(v_pages);
  p.page_size = page_size;
  p.heads = Hkv;
  p.D = D;
  const cudaError_t e = dash::launch_cache_copy(p, pairs.data(), n, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "cache copy launch");
} catch (...) {
  return report(DASH_ERR_NO_MEMORY, "cache copy: out of host memory");
}

}  // extern "C"
