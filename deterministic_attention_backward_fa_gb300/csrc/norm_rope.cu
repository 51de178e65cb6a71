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
constexpr int kAhead = 4;     // head rows that a lane has in flight, forward
constexpr int kAheadBwd = 4;  // and backward (x and dz)

// Two 32-bit values; the arithmetic is one instruction for both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 parts(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator-(F2 a) { return a * f2(-1.f, -1.f); }

// A lane's eight values of a row as pairs (a[i], b[i]), i < 4.
struct Eight {
  F2 a[2], b[2];
};

// What a lane holds of a head row.
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
  static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ Eight widen(const uint2 (&w)[2]) {
    Eight x;
    if (kPairs) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.a[i] = f2(low(w[i].x), low(w[i].y));
        x.b[i] = f2(high(w[i].x), high(w[i].y));
      }
    } else {
      x.a[0] = f2(low(w[0].x), high(w[0].x));
      x.a[1] = f2(low(w[0].y), high(w[0].y));
      x.b[0] = f2(low(w[1].x), high(w[1].x));
      x.b[1] = f2(low(w[1].y), high(w[1].y));
    }
    return x;
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, const Eight &x) const {
    uint2 w[2];
    const float2 a0 = parts(x.a[0]), a1 = parts(x.a[1]), b0 = parts(x.b[0]), b1 = parts(x.b[1]);
    if (kPairs) {
      w[0] = make_uint2(pack_bf16(a0.x, b0.x), pack_bf16(a0.y, b0.y));
      w[1] = make_uint2(pack_bf16(a1.x, b1.x), pack_bf16(a1.y, b1.y));
    } else {
      w[0] = make_uint2(pack_bf16(a0.x, a0.y), pack_bf16(a1.x, a1.y));
      w[1] = make_uint2(pack_bf16(b0.x, b0.y), pack_bf16(b1.x, b1.y));
    }
    *reinterpret_cast<uint2 *>(row + lo) = w[0];
    *reinterpret_cast<uint2 *>(row + hi) = w[1];
  }
  __device__ __forceinline__ Eight weight(const NormRopeParams &p, int which) const {
    if (!p.weight32) {
      uint2 w[2];
      load(static_cast<const __nv_bfloat16 *>(p.t[which].weight), w);
      return widen(w);
    }
    const float *w = static_cast<const float *>(p.t[which].weight);
    const float4 u = *reinterpret_cast<const float4 *>(w + lo), v = *reinterpret_cast<const float4 *>(w + hi);
    Eight x;
    if (kPairs) {
      x.a[0] = f2(u.x, u.z), x.a[1] = f2(v.x, v.z);
      x.b[0] = f2(u.y, u.w), x.b[1] = f2(v.y, v.w);
    } else {
      x.a[0] = f2(u.x, u.y), x.a[1] = f2(u.z, u.w);
      x.b[0] = f2(v.x, v.y), x.b[1] = f2(v.z, v.w);
    }
    return x;
  }
  // Cosines (a) and sines (b) of a row's position; NaN, and a report, where it is outside the table.
  __device__ __forceinline__ Eight angles(const NormRopeParams &p, long long row, int lane) const {
    const int pos = p.positions[row];
    const bool ok = pos >= 0 && pos < p.max_positions;
    Eight x;
    if (ok && angle >= 0) {
      const float *t = p.rope + (long long)pos * p.rot + angle;
      const float4 c = __ldg(reinterpret_cast<const float4 *>(t));
      const float4 s = __ldg(reinterpret_cast<const float4 *>(t + p.rot / 2));
      x.a[0] = f2(c.x, c.y), x.a[1] = f2(c.z, c.w);
      x.b[0] = f2(s.x, s.y), x.b[1] = f2(s.z, s.w);
    } else {
      if (!ok && lane == 0) atomicCAS(p.status, 0, kStatusBadPosition);
      x.a[0] = x.a[1] = ok ? f2(1.f, 1.f) : f2(NAN, NAN);
      x.b[0] = x.b[1] = ok ? f2(0.f, 0.f) : f2(NAN, NAN);
    }
    return x;
  }
  static __device__ __forceinline__ float sum(F2 x) {
    const float2 v = parts(x);
    float s = v.x + v.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
};

// Steps first .. end - 1 of a tensor's heads for one row of the batch, with
// w cos, w sin made once: z_a = r (x_a (w_a cos) - x_b (w_b sin)) and so on.
template <int D, bool kPairs>
__device__ __forceinline__ void norm_heads(const NormRopeParams &p, const Lane<D, kPairs> &l, int which, long long row,
                                           const Eight &angle, int lane, int first, int end) {
  using L = Lane<D, kPairs>;
  const NormRopeTensor &t = p.t[which];
  const int sub = lane / L::kLanes;
  const __nv_bfloat16 *in = t.x + row * t.x_row + (first * L::kRows + sub) * t.x_head;
  __nv_bfloat16 *out = t.out + row * t.out_row + (first * L::kRows + sub) * t.out_head;
  const long long in_step = L::kRows * t.x_head, out_step = L::kRows * t.out_head;
  F2 ac[2], bs[2], bc[2], as[2];
  const Eight w = l.weight(p, which);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ac[i] = w.a[i] * angle.a[i];
    bs[i] = -(w.b[i] * angle.b[i]);
    bc[i] = w.b[i] * angle.a[i];
    as[i] = w.a[i] * angle.b[i];
  }
  for (int s0 = first; s0 < end; s0 += kAhead) {
    uint2 x[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      x[u][0] = x[u][1] = make_uint2(0u, 0u);
      if (s0 + u < end && (s0 + u) * L::kRows + sub < t.heads) l.load(in + u * in_step, x[u]);
    }
    in += kAhead * in_step;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s0 + u >= end) break;
      const Eight v = L::widen(x[u]);
      F2 sq = v.a[0] * v.a[0];
      sq = fma(v.a[1], v.a[1], sq);
      sq = fma(v.b[0], v.b[0], sq);
      sq = fma(v.b[1], v.b[1], sq);
      const float r = rsqrtf(L::sum(sq) * (1.f / D) + p.eps);
      const F2 rr = f2(r, r);
      Eight z;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        z.a[i] = rr * fma(v.a[i], ac[i], v.b[i] * bs[i]);
        z.b[i] = rr * fma(v.b[i], bc[i], v.a[i] * as[i]);
      }
      if ((s0 + u) * L::kRows + sub < t.heads) l.store(out, z);
      out += out_step;
    }
  }
}

// A warp takes one row of the batch and `passes` steps of its heads, the queries' first.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) dash_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // below 2^31: many rows are a warp each
  const unsigned at_row = item / (unsigned)p.blocks;
  if (at_row >= p.rows) return;
  const int first = (int)(item - at_row * p.blocks) * p.passes;
  const L l(lane, p.rot);
  const int q_steps = (p.t[0].heads + L::kRows - 1) / L::kRows, k_steps = (p.t[1].heads + L::kRows - 1) / L::kRows;
  const int end = min(first + p.passes, q_steps + k_steps);
  const Eight angle = l.angles(p, at_row, lane);
  if (first < q_steps) norm_heads(p, l, 0, at_row, angle, lane, first, min(end, q_steps));
  if (end > q_steps) norm_heads(p, l, 1, at_row, angle, lane, max(first - q_steps, 0), end - q_steps);
}

// A warp takes rows of the batch in turn and keeps its sums of dw in registers.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2) dash_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  constexpr int kWarps = kThreads / 32;
  // the sum of the parts may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L::kLanes;
  const L l(lane, p.rot);
  Eight w[2], dw[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    w[which] = l.weight(p, which);
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[which].a[i] = dw[which].b[i] = f2(0.f, 0.f);
  }
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows; row += (long long)gridDim.x * kWarps) {
    const Eight angle = l.angles(p, row, lane);
    F2 minus[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) minus[i] = -angle.b[i];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const NormRopeTensor &t = p.t[which];
      const __nv_bfloat16 *xs = t.x + row * t.x_row + sub * t.x_head, *zs = t.dz + row * t.dz_row + sub * t.dz_head;
      __nv_bfloat16 *out = t.out + row * t.out_row + sub * t.out_head;
      for (int h0 = 0; h0 < t.heads; h0 += kAheadBwd * L::kRows) {
        uint2 xw[kAheadBwd][2], zw[kAheadBwd][2];
#pragma unroll
        for (int u = 0; u < kAheadBwd; ++u) {
          xw[u][0] = xw[u][1] = zw[u][0] = zw[u][1] = make_uint2(0u, 0u);
          if (h0 + u * L::kRows + sub < t.heads) {
            l.load(xs + (h0 + u * L::kRows) * t.x_head, xw[u]);
            l.load(zs + (h0 + u * L::kRows) * t.dz_head, zw[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < kAheadBwd; ++u) {
          if (h0 + u * L::kRows >= t.heads) break;
          const Eight x = L::widen(xw[u]), z = L::widen(zw[u]);
          Eight g, gw;
          F2 sq = f2(0.f, 0.f), dot = f2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            g.a[i] = fma(z.a[i], angle.a[i], z.b[i] * angle.b[i]);
            g.b[i] = fma(z.b[i], angle.a[i], z.a[i] * minus[i]);
            gw.a[i] = g.a[i] * w[which].a[i];
            gw.b[i] = g.b[i] * w[which].b[i];
            sq = fma(x.a[i], x.a[i], sq);
            sq = fma(x.b[i], x.b[i], sq);
            dot = fma(gw.a[i], x.a[i], dot);
            dot = fma(gw.b[i], x.b[i], dot);
          }
          // lanes past the last head hold zeros: their r is 0, so that they add nothing to dw whatever eps is
          const bool real = h0 + u * L::kRows + sub < t.heads;
          const float var = L::sum(sq) * (1.f / D) + p.eps, r = real ? rsqrtf(var) : 0.f;
          const float m = -(L::sum(dot) * (1.f / D) * r * r * r);
          const F2 rr = f2(r, r), mm = f2(m, m);
          Eight d;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            d.a[i] = fma(gw.a[i], rr, x.a[i] * mm);
            d.b[i] = fma(gw.b[i], rr, x.b[i] * mm);
            dw[which].a[i] = fma(g.a[i], x.a[i] * rr, dw[which].a[i]);
            dw[which].b[i] = fma(g.b[i], x.b[i] * rr, dw[which].b[i]);
          }
          if (real) l.store(out + (h0 + u * L::kRows) * t.out_head, d);
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
      const float2 va = parts(dw[which].a[i / 2]), vb = parts(dw[which].b[i / 2]);
      float a = i & 1 ? va.y : va.x, b = i & 1 ? vb.y : vb.x;
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
  const int steps = (p.t[0].heads + kRows - 1) / kRows + (p.t[1].heads + kRows - 1) / kRows;
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
