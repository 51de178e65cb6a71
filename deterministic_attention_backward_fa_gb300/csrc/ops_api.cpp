// C ABI of the operators around the attention (declared in include/dash.h): the
// norms of queries and keys with their rotation, and the decode of a batch that
// shares a prefix.
#include "norm_rope.h"
#include "ops_host.h"
#include "shared.h"

using dash::report;
using namespace dash::host;

namespace {

// What the norms' forward and backward have in common; `p` gets all but the pointers of the outputs.
dash_status_t norm_params(const void *q_weight, const void *k_weight, int weight_fp32, const float *rope,
                          const int32_t *positions, long long rows, int Hq, int Hkv, int D, int rot,
                          int max_positions, int pairs, float eps, dash::NormRopeParams *p) {
  dash_status_t st;
  if (D != 64 && D != 128) return report(DASH_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", D);
  if (Hq < 1 || Hkv < 1) return report(DASH_ERR_INVALID_ARG, "q and k need heads");
  if (Hq > 65535 || Hkv > 65535) return report(DASH_ERR_UNSUPPORTED, "more than 65535 heads");
  if (rot < 8 || rot > D || rot % 8)
    return report(DASH_ERR_INVALID_ARG, "rot = %d must be a multiple of 8 of at most D", rot);
  if (max_positions < 1) return report(DASH_ERR_INVALID_ARG, "the rotation table needs positions");
  if (rows < 0) return report(DASH_ERR_INVALID_ARG, "rows must be >= 0");
  if (rows > INT32_MAX - 65536) return report(DASH_ERR_UNSUPPORTED, "more than 2^31 rows");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return report(DASH_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((st = check_ptr(q_weight, "q_weight")) || (st = check_ptr(k_weight, "k_weight")) ||
      (st = check_ptr(rope, "rope")) || (st = check_words(positions, "positions", rows == 0)))
    return st;
  p->t[0].weight = q_weight;
  p->t[1].weight = k_weight;
  p->t[0].heads = Hq;
  p->t[1].heads = Hkv;
  p->rope = rope;
  p->positions = positions;
  p->rows = rows;
  p->D = D;
  p->rot = rot;
  p->max_positions = max_positions;
  p->weight32 = weight_fp32 != 0;
  p->pairs = pairs != 0;
  p->eps = eps;
  return DASH_OK;
}

dash_status_t norm_rows(const int64_t *strides, int i, const void *ptr, long long rows, int heads, int D,
                        const char *name, long long *row, long long *head) {
  Rows r;
  dash_status_t st;
  if ((st = check_ptr(ptr, name)) || (st = rows_of(strides, i, rows, heads, D, name, &r))) return st;
  *row = r.row;
  *head = r.head;
  return DASH_OK;
}

}  // namespace

extern "C" {

dash_status_t dash_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const void *q_weight,
                                const void *k_weight, int weight_fp32, const float *rope, const int32_t *positions,
                                long long rows, int Hq, int Hkv, int D, int rot, int max_positions, int pairs,
                                float eps, const int64_t *strides, dash_stream_t stream) {
  dash::NormRopeParams p = {};
  dash_status_t st = norm_params(q_weight, k_weight, weight_fp32, rope, positions, rows, Hq, Hkv, D, rot,
                                 max_positions, pairs, eps, &p);
  if (st != DASH_OK || rows == 0) return st;
  const void *in[2] = {q, k};
  void *out[2] = {q_out, k_out};
  const char *names[4] = {"q", "k", "q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    dash::NormRopeTensor &t = p.t[i];
    if ((st = norm_rows(strides, i, in[i], rows, t.heads, D, names[i], &t.x_row, &t.x_head)) ||
        (st = norm_rows(strides, 2 + i, out[i], rows, t.heads, D, names[2 + i], &t.out_row, &t.out_head)))
      return st;
    t.x = static_cast<const __nv_bfloat16 *>(in[i]);
    t.out = static_cast<__nv_bfloat16 *>(out[i]);
  }
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  const cudaError_t e = dash::launch_norm_rope(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "norm launch");
}

long long dash_norm_rope_workspace(long long rows, int Hq, int Hkv, int D) {
  if (rows < 0 || rows > INT32_MAX || Hq < 1 || Hkv < 1 || Hq > 65535 || Hkv > 65535 || (D != 64 && D != 128)) return -1;
  return (long long)dash::norm_bwd_ctas(dash::norm_steps(rows, Hq, Hkv, D)) * 2 * D * 4;
}

dash_status_t dash_qk_norm_rope_bwd(const void *q, const void *k, const void *dq_out, const void *dk_out, void *dq,
                                    void *dk, const void *q_weight, const void *k_weight, int weight_fp32,
                                    float *dq_weight, float *dk_weight, const float *rope, const int32_t *positions,
                                    long long rows, int Hq, int Hkv, int D, int rot, int max_positions, int pairs,
                                    float eps, const int64_t *strides, void *workspace, long long workspace_bytes,
                                    dash_stream_t stream) {
  dash::NormRopeParams p = {};
  dash_status_t st = norm_params(q_weight, k_weight, weight_fp32, rope, positions, rows, Hq, Hkv, D, rot,
                                 max_positions, pairs, eps, &p);
  if (st != DASH_OK) return st;
  if ((st = check_words(dq_weight, "dq_weight")) || (st = check_words(dk_weight, "dk_weight"))) return st;
  const void *in[2] = {q, k}, *dz[2] = {dq_out, dk_out};
  void *out[2] = {dq, dk};
  const char *names[6] = {"q", "k", "dq_out", "dk_out", "dq", "dk"};
  for (int i = 0; i < 2; ++i) {
    dash::NormRopeTensor &t = p.t[i];
    t.dweight = i ? dk_weight : dq_weight;
    if (rows == 0) continue;
    if ((st = norm_rows(strides, i, in[i], rows, t.heads, D, names[i], &t.x_row, &t.x_head)) ||
        (st = norm_rows(strides, 2 + i, dz[i], rows, t.heads, D, names[2 + i], &t.dz_row, &t.dz_head)) ||
        (st = norm_rows(strides, 4 + i, out[i], rows, t.heads, D, names[4 + i], &t.out_row, &t.out_head)))
      return st;
    t.x = static_cast<const __nv_bfloat16 *>(in[i]);
    t.dz = static_cast<const __nv_bfloat16 *>(dz[i]);
    t.out = static_cast<__nv_bfloat16 *>(out[i]);
  }
  const long long need = dash_norm_rope_workspace(rows, Hq, Hkv, D);
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need))
    return report(DASH_ERR_INVALID_ARG, "the workspace must hold %lld bytes, 16-byte aligned", need);
  p.parts = static_cast<float *>(workspace);
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  const cudaError_t e = dash::launch_norm_rope_bwd(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "norm backward launch");
}

long long dash_decode_shared_workspace(int B, int Hq, int Hkv, int D, int page_size, int max_pages, int prefix) {
  if (prefix == 0) return dash_decode_workspace(B, Hq, D, page_size, max_pages);
  if (B < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || (D != 64 && D != 128) || page_size < 1 || max_pages < 0 || prefix < 0 ||
      (long long)page_size * max_pages > kMaxCached || prefix > (long long)page_size * max_pages)
    return -1;
  if (dash::prefix_with_tails(B, Hq, Hkv, page_size * max_pages))
    return dash_decode_workspace(B, Hq, D, page_size, max_pages);
  const int parts = dash::prefix_cut(std::max(B, 1), Hq, Hkv, prefix).splits +
                    std::max(1, dash::decode_max_splits(page_size * max_pages - prefix));
  return (long long)B * Hq * parts * (D * 4 + 8) + 256;
}

dash_status_t dash_attn_decode_shared(const void *q, const void *k_pages, const void *v_pages,
                                      const int32_t *page_table, const int32_t *lengths, int prefix, void *o,
                                      float *lse, int B, int Hq, int Hkv, int D, int n_pages, int page_size,
                                      int max_pages, const int64_t *strides, float scale, void *workspace,
                                      long long workspace_bytes, dash_stream_t stream) {
  if (prefix < 0 || (page_size > 0 && max_pages >= 0 && prefix > (long long)page_size * max_pages))
    return report(DASH_ERR_INVALID_ARG, "a prefix of %d tokens does not fit %d pages of %d", prefix, max_pages,
                  page_size);
  if (prefix == 0)
    return dash_attn_decode(q, k_pages, v_pages, page_table, lengths, o, lse, B, Hq, Hkv, D, n_pages, page_size,
                            max_pages, strides, scale, workspace, workspace_bytes, stream);
  dash_status_t st = check_heads(Hq, Hkv, D);
  if (st != DASH_OK) return st;
  if ((long long)B * (Hq / Hkv) > 65535LL * 2 * dash::kPackedTile)
    return report(DASH_ERR_UNSUPPORTED, "more than %lld rows on one K/V head", 65535LL * 2 * dash::kPackedTile);
  dash::SharedParams p = {};
  const dash::PrefixCut cut = dash::prefix_cut(std::max(B, 1), Hq, Hkv, prefix);
  const bool together = max_pages >= 0 && page_size > 0 && (long long)page_size * max_pages <= kMaxCached && B >= 0 &&
                        dash::prefix_with_tails(B, Hq, Hkv, page_size * max_pages);
  if ((st = decode_params(q, page_table, lengths, o, lse, B, Hq, Hkv, D, n_pages, page_size, max_pages, strides,
                          strides ? strides + 10 : nullptr, scale, workspace, workspace_bytes,
                          dash_decode_shared_workspace(B, Hq, Hkv, D, page_size, max_pages, prefix),
                          together ? 0 : prefix, together ? 0 : cut.splits, &p)) != DASH_OK ||
      B == 0)
    return st;
  if ((st = decode_cache(k_pages, v_pages, Hkv, D, n_pages, page_size, strides, &p)) != DASH_OK) return st;
  p.prefix_tiles = (prefix + dash::kPackedTile - 1) / dash::kPackedTile;
  p.tiles_per_split = cut.tiles;
  p.spin_limit_ns = kSpinNs;
  int dev = 0;
  Device device;
  if ((st = current_device(&dev, &device)) != DASH_OK) return st;
  p.status = device.status;
  p.shared = together ? prefix : 0;
  const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = together ? dash::launch_decode(D, p, device.sms, on)
                                 : dash::launch_decode_shared(D, p, device.sms, on);
  return e == cudaSuccess ? DASH_OK : cuda_error(e, "decode launch");
}

}  // extern "C"
