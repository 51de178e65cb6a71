// Norms of queries and keys with their rotation by position: what the entry
// points (ops_api.cpp) and the kernels (norm_rope.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace dash {

// One of the two tensors of a call: rows of x (and dz), what is written, and the weight.
struct NormRopeTensor {
  const __nv_bfloat16 *x, *dz;
  __nv_bfloat16 *out;          // z, or dx in the backward
  long long x_row, x_head, dz_row, dz_head, out_row, out_head;
  const void *weight;          // [D], bf16 or fp32
  float *dweight;              // [D]
  int heads;
};

struct NormRopeParams {
  NormRopeTensor t[2];         // queries, keys
  const float *rope;           // [max_positions][rot]: rot / 2 cosines, then rot / 2 sines
  const int *positions;        // [rows]
  float *parts;                // backward: [CTA][2][D], the weights' gradients of the CTA's rows
  long long rows;
  int D, rot, max_positions;
  int blocks, passes;          // forward: a row's heads are dealt to `blocks` warps, `passes` steps each
  long long steps, per_warp;   // backward: of the call, of a warp
  bool weight32, pairs;
  float eps;
  int *status;
};

// Steps of a call: 512 bytes of a row's queries or of its keys each.
inline long long norm_steps(long long rows, int Hq, int Hkv, int D) {
  const int n = 256 / D;
  return rows * ((Hq + n - 1) / n + (Hkv + n - 1) / n);
}
// CTAs of a backward: a number of its own for each size, whatever the GPU, so
// that the weights' gradients are the same sums everywhere.
constexpr int kNormBwdCtas = 304;
inline int norm_bwd_ctas(long long steps) {
  return steps < 8LL * kNormBwdCtas ? (int)((steps + 7) / 8) : kNormBwdCtas;
}

cudaError_t prepare_norm_rope();
cudaError_t launch_norm_rope(NormRopeParams p, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(NormRopeParams p, cudaStream_t stream);

}  // namespace dash
