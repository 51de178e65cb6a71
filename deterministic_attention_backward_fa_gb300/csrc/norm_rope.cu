// Norms of queries and keys, head by head, and their rotation by position, in
// one pass; and its backward.  Per row x of D values at position s:
//   r = (mean x^2 + eps)^-1/2,  y = w (x r),
//   z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin
// for each pair (a, b) of the first `rot` values, with the pair's angle at s;
// the values behind them are only normed.  Backward, with g = dz turned back by
// the same angles:
//   dx = r (g w - x r^2 mean(g w x)),   dw = sum over rows and heads of g x r.
// All in 32 bits; rounded to bf16 once, when z or dx is written.
//
// Bound by bytes: 2 + 2 a value forward, 4 + 2 backward.  A row is D / 8 lanes:
// a lane holds both sides of four pairs (4 values at `a`, 4 at `b`, 8 bytes
// each), so that the rotation needs no exchange and every lane reads the four
// cosines and sines that it needs, once for all heads of a row of the batch.
#include <cuda_runtime.h>

#include "norm_rope.h"
#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // head rows that a lane has in flight

__device__ __forceinline__ void widen(uint2 w, float *v) {
  v[0] = __uint_as_float(w.x << 16);
  v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16);
  v[3] = __uint_as_float(w.y & 0xffff0000u);
}

// What a lane holds of a head row: its eight values as pairs (a[i], b[i]).
template <int D, bool kPairs>
struct Lane {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a head row, head rows of a warp's step
  int lo, hi;   // offsets of its two runs of four values
  int angle;    // its first angle; -1: it is not turned

  __device__ __forceinline__ Lane(int lane, int rot) {
    const int c = lane % kLanes;
    if (kPairs) {  // neighbours are pairs
      lo = 8 * c;
      hi = lo + 4;
      angle = lo < rot ? 4 * c : -1;
    } else {       // value i and value rot / 2 + i are a pair
      const bool turned = 8 * c < rot;
      const int half = turned ? rot / 2 : (D - rot) / 2, first = turned ? 4 * c : rot + 4 * (c - rot / 8);
      lo = first;
      hi = first + half;
      angle = turned ? first : -1;
    }
  }
  __device__ __forceinline__ void load(const __nv_bfloat16 *row, uint2 (&w)[2]) const {
    w[0] = *reinterpret_cast<const uint2 *>(row + lo);
    w[1] = *reinterpret_cast<const uint2 *>(row + hi);
  }
  static __device__ __forceinline__ void split(const uint2 (&w)[2], float (&a)[4], float (&b)[4]) {
    float v[8];
    widen(w[0], v);
    widen(w[1], v + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = kPairs ? v[2 * i] : v[i];
      b[i] = kPairs ? v[2 * i + 1] : v[4 + i];
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, const float (&a)[4], const float (&b)[4]) const {
    uint2 w[2];
    if (kPairs) {
      w[0] = make_uint2(pack_bf16(a[0], b[0]), pack_bf16(a[1], b[1]));
      w[1] = make_uint2(pack_bf16(a[2], b[2]), pack_bf16(a[3], b[3]));
    } else {
      w[0] = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
      w[1] = make_uint2(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]));
    }
    *reinterpret_cast<uint2 *>(row + lo) = w[0];
    *reinterpret_cast<uint2 *>(row + hi) = w[1];
  }
  __device__ __forceinline__ void weight(const NormRopeParams &p, int which, float (&a)[4], float (&b)[4]) const {
    float v[8];
    if (p.weight32) {
      const float *w = static_cast<const float *>(p.t[which].weight);
      *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(w + lo);
      *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(w + hi);
    } else {
      uint2 w[2];
      load(static_cast<const __nv_bfloat16 *>(p.t[which].weight), w);
      widen(w[0], v);
      widen(w[1], v + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = kPairs ? v[2 * i] : v[i];
      b[i] = kPairs ? v[2 * i + 1] : v[4 + i];
    }
  }
  // Cosines and sines of a row's position.  False: the position is outside the table.
  __device__ __forceinline__ bool angles(const NormRopeParams &p, long long row, float (&c)[4], float (&s)[4]) const {
    const int pos = p.positions[row];
    const bool ok = pos >= 0 && pos < p.max_positions;
    if (ok && angle >= 0) {
      const float *t = p.rope + (long long)pos * p.rot + angle;
      *reinterpret_cast<float4 *>(c) = __ldg(reinterpret_cast<const float4 *>(t));
      *reinterpret_cast<float4 *>(s) = __ldg(reinterpret_cast<const float4 *>(t + p.rot / 2));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
    return ok;
  }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp takes one row of the batch and `passes` steps of its heads.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) dash_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // below 2^31: many rows are a warp each
  const unsigned at_row = item / (unsigned)p.blocks;
  if (at_row >= p.rows) return;
  const int first = (int)(item - at_row * p.blocks) * p.passes;
  const long long row = at_row;
  const L l(lane, p.rot);
  const int heads = p.t[0].heads + p.t[1].heads;
  const int sub = lane / L::kLanes;
  float wa[2][4], wb[2][4], c[4], s[4];
  uint2 x[kAhead][2];
  auto at = [&](int pass, int &which, int &h) {
    h = (first + pass) * L::kRows + sub;
    which = h >= p.t[0].heads;
    const bool valid = pass < p.passes && h < heads;
    if (which) h -= p.t[0].heads;
    return valid;
  };
  auto load = [&](int pass0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      int which, h;
      x[u][0] = x[u][1] = make_uint2(0u, 0u);
      if (at(pass0 + u, which, h)) l.load(p.t[which].x + row * p.t[which].x_row + h * p.t[which].x_head, x[u]);
    }
  };
  load(0);
  const bool ok = l.angles(p, row, c, s);
  if (!ok && lane == 0) atomicCAS(p.status, 0, kStatusBadPosition);
  l.weight(p, 0, wa[0], wb[0]);
  l.weight(p, 1, wa[1], wb[1]);
  for (int pass0 = 0; pass0 < p.passes; pass0 += kAhead) {
    if (pass0) load(pass0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float a[4], b[4], sum = 0.f;
      l.split(x[u], a, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
      const float r = ok ? rsqrtf(row_sum<L::kLanes>(sum) * (1.f / D) + p.eps) : NAN;
      int which, h;
      if (!at(pass0 + u, which, h)) continue;
      float za[4], zb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ya = a[i] * r * (which ? wa[1][i] : wa[0][i]), yb = b[i] * r * (which ? wb[1][i] : wb[0][i]);
        za[i] = ya * c[i] - yb * s[i];
        zb[i] = yb * c[i] + ya * s[i];
      }
      l.store(p.t[which].out + row * p.t[which].out_row + h * p.t[which].out_head, za, zb);
    }
  }
}

// A warp takes rows of the batch in turn and keeps its sums of dw in registers.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) dash_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  constexpr int kWarps = kThreads / 32;
  // the sum of the parts may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L::kLanes;
  const L l(lane, p.rot);
  float dwa[2][4] = {}, dwb[2][4] = {};
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const NormRopeTensor &t = p.t[which];
    float wa[4], wb[4];
    l.weight(p, which, wa, wb);
    for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows; row += (long long)gridDim.x * kWarps) {
      float c[4], s[4];
      const bool ok = l.angles(p, row, c, s);
      if (!ok && lane == 0) atomicCAS(p.status, 0, kStatusBadPosition);
      for (int h0 = 0; h0 < t.heads; h0 += 2 * L::kRows) {
        uint2 xw[2][2], gw[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int h = h0 + u * L::kRows + sub;
          xw[u][0] = xw[u][1] = gw[u][0] = gw[u][1] = make_uint2(0u, 0u);
          if (h < t.heads) {
            l.load(t.x + row * t.x_row + h * t.x_head, xw[u]);
            l.load(t.dz + row * t.dz_row + h * t.dz_head, gw[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int h = h0 + u * L::kRows + sub;
          float a[4], b[4], za[4], zb[4], ga[4], gb[4], sum = 0.f, dot = 0.f;
          l.split(xw[u], a, b);
          l.split(gw[u], za, zb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ga[i] = za[i] * c[i] + zb[i] * s[i];
            gb[i] = zb[i] * c[i] - za[i] * s[i];
            sum += a[i] * a[i] + b[i] * b[i];
            dot += ga[i] * wa[i] * a[i] + gb[i] * wb[i] * b[i];
          }
          sum = row_sum<L::kLanes>(sum);
          dot = row_sum<L::kLanes>(dot);
          if (h >= t.heads) continue;
          const float r = ok ? rsqrtf(sum * (1.f / D) + p.eps) : NAN;
          const float m = dot * (1.f / D) * r * r;
          float xa[4], xb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xa[i] = r * (ga[i] * wa[i] - a[i] * m);
            xb[i] = r * (gb[i] * wb[i] - b[i] * m);
            dwa[which][i] += ga[i] * (a[i] * r);
            dwb[which][i] += gb[i] * (b[i] * r);
          }
          l.store(t.out + row * t.out_row + h * t.out_head, xa, xb);
        }
      }
    }
  }
  // the CTA's sums: lanes that hold the same values, then warps, in their order
  __shared__ float s_dw[kWarps][2][D];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = dwa[which][i], b = dwb[which][i];
#pragma unroll
      for (int o = L::kLanes; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (sub == 0) {
        s_dw[warp][which][kPairs ? l.lo + 2 * i : l.lo + i] = a;
        s_dw[warp][which][kPairs ? l.lo + 2 * i + 1 : l.hi + i] = b;
      }
    }
  __syncthreads();
  for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += (&s_dw[w][0][0])[x];
    p.parts[(long long)blockIdx.x * 2 * D + x] = sum;
  }
}

// dw from the CTAs' sums: a CTA takes 8 of the 2 D columns, 32 threads a column,
// each every 32nd part; then their sums in one order.
__global__ void __launch_bounds__(256) dash_norm_rope_sum_kernel(const __grid_constant__ NormRopeParams p, int n) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), part = threadIdx.x >> 3;
  float sum = 0.f;
#pragma unroll 4
  for (int i = part; i < n; i += 32) sum += p.parts[(long long)i * 2 * p.D + col];
  __shared__ float s_sum[32][8];
  s_sum[part][threadIdx.x & 7] = sum;
  __syncthreads();
  if (part == 0) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s_sum[i][threadIdx.x];
    (col < p.D ? p.t[0].dweight : p.t[1].dweight - p.D)[col] = sum;
  }
}

template <int D>
cudaError_t launch_fwd(NormRopeParams &p, cudaStream_t stream) {
  constexpr int kRows = 256 / D;
  const int steps = (p.t[0].heads + p.t[1].heads + kRows - 1) / kRows;
  // Rows enough to fill the GPU are a warp each, which reads a row's angles once;
  // of few rows, a warp takes a part of the heads.
  const long long want = 4096;
  p.blocks = p.rows >= want ? 1 : (int)((want + p.rows - 1) / p.rows);
  if (p.blocks > steps) p.blocks = steps;
  p.passes = (steps + p.blocks - 1) / p.blocks;
  p.blocks = (steps + p.passes - 1) / p.passes;
  const long long warps = p.rows * p.blocks;
  return launch(p.pairs ? dash_norm_rope_kernel<D, true> : dash_norm_rope_kernel<D, false>,
                dim3((unsigned)((warps + 7) / 8)), kThreads, 0, stream, nullptr, p);
}

template <int D>
cudaError_t launch_bwd(const NormRopeParams &p, cudaStream_t stream) {
  const int ctas = norm_bwd_ctas(p.rows);  // 0 without rows: dw is then a sum of nothing
  cudaError_t e = ctas == 0 ? cudaSuccess : launch(p.pairs ? dash_norm_rope_bwd_kernel<D, true> : dash_norm_rope_bwd_kernel<D, false>, ctas,
                         kThreads, 0, stream, nullptr, p);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = overlap_attr();
  return launch(dash_norm_rope_sum_kernel, 2 * D / 8, 256, 0, stream, &attr, p, ctas);
}

template <int D>
cudaError_t prepare_t() {
  cudaFuncAttributes fa;
  for (auto kernel : {dash_norm_rope_kernel<D, true>, dash_norm_rope_kernel<D, false>,
                      dash_norm_rope_bwd_kernel<D, true>, dash_norm_rope_bwd_kernel<D, false>})
    if (const cudaError_t e = cudaFuncGetAttributes(&fa, kernel)) return e;
  return cudaFuncGetAttributes(&fa, dash_norm_rope_sum_kernel);
}

}  // namespace

cudaError_t prepare_norm_rope() {
  const cudaError_t e = prepare_t<64>();
  return e != cudaSuccess ? e : prepare_t<128>();
}

cudaError_t launch_norm_rope(NormRopeParams p, cudaStream_t stream) {
  return p.D == 64 ? launch_fwd<64>(p, stream) : launch_fwd<128>(p, stream);
}

cudaError_t launch_norm_rope_bwd(NormRopeParams p, cudaStream_t stream) {
  return p.D == 64 ? launch_bwd<64>(p, stream) : launch_bwd<128>(p, stream);
}

}  // namespace dash
