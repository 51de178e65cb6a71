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
// each), so that the rotation needs no exchange and every lane holds the four
// cosines and sines that it needs, once for all heads of a row of the batch.
// 16384 tokens of 16 + 4 heads of 128: 31.4 us forward and 48.1 us backward, 5.4
// and 5.3 TB/s.  Next to the bytes stand the instructions (130 and 213 a step
// of 32 lanes x 8 values): forward, loads straight into registers and two steps'
// arithmetic side by side beat a ring in shared memory (35.1 us); backward,
// where registers hold the sums of dw too, the ring wins (53.3 us without it).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "norm_rope.h"
#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;   // steps that a lane has in flight beside those at hand, forward (4 on 3 CTAs of an SM: the same)
constexpr int kStages = 6;  // steps of a warp that are in flight, backward (4: the same, 8: 2 % slower)

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
    if (kPairs) {
      const uint4 u = *reinterpret_cast<const uint4 *>(row + lo);
      w[0] = make_uint2(u.x, u.y);
      w[1] = make_uint2(u.z, u.w);
    } else {
      w[0] = *reinterpret_cast<const uint2 *>(row + lo);
      w[1] = *reinterpret_cast<const uint2 *>(row + hi);
    }
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
  // Cosines (a) and sines (b) of a row, from its part of the table; NaN where its position is outside.
  __device__ __forceinline__ Eight angles(const float *t, int rot, bool ok) const {
    Eight x;
    if (ok && angle >= 0) {
      const float4 c = *reinterpret_cast<const float4 *>(t + angle);
      const float4 s = *reinterpret_cast<const float4 *>(t + rot / 2 + angle);
      x.a[0] = f2(c.x, c.y), x.a[1] = f2(c.z, c.w);
      x.b[0] = f2(s.x, s.y), x.b[1] = f2(s.z, s.w);
    } else {
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

// A warp takes one row of the batch and `passes` steps of its heads, the queries'
// first, kAhead at a time; the next ones' loads are under way by then.  w cos
// and w sin are made once for the queries and once for the keys:
// z_a = r (x_a (w_a cos) - x_b (w_b sin)) and so on.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) dash_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  const int lane = threadIdx.x & 31, sub = lane / L::kLanes;
  const unsigned item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // below 2^31: many rows are a warp each
  const unsigned row = item / (unsigned)p.blocks;
  if (row >= p.rows) return;
  const int pos = p.positions[row];
  const int q_steps = (p.t[0].heads + L::kRows - 1) / L::kRows, k_steps = (p.t[1].heads + L::kRows - 1) / L::kRows;
  const int first = (int)(item - row * p.blocks) * p.passes, end = min(first + p.passes, q_steps + k_steps);
  const L l(lane, p.rot);
  // steps s .. of one tensor
  auto load = [&](int s, uint2 (&x)[kAhead][2]) {
    const bool k = s >= q_steps;
    const NormRopeTensor &t = p.t[k];
    int h = (k ? s - q_steps : s) * L::kRows + sub;
    const __nv_bfloat16 *in = t.x + row * t.x_row + h * t.x_head;
    const long long by = L::kRows * t.x_head;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      x[u][0] = x[u][1] = make_uint2(0u, 0u);
      if (s + u < end && h < t.heads) l.load(in, x[u]);
      in += by;
      h += L::kRows;
    }
  };
  uint2 x[kAhead][2], ahead[kAhead][2];
  load(first, x);
  const bool ok = pos >= 0 && pos < p.max_positions;
  if (!ok && lane == 0) atomicCAS(p.status, 0, kStatusBadPosition);
  const Eight angle = l.angles(p.rope + (ok ? (long long)pos * p.rot : 0), p.rot, ok);
  F2 ac[2], bs[2], bc[2], as[2];
  for (int s = first, next; s < end; s = next) {
    const bool k = s >= q_steps;
    const NormRopeTensor &t = p.t[k];
    next = min(s + kAhead, k ? end : min(end, q_steps));
    if (next < end) load(next, ahead);
    if (s == first || s == q_steps) {
      const Eight w = l.weight(p, k);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ac[i] = w.a[i] * angle.a[i];
        bs[i] = -(w.b[i] * angle.b[i]);
        bc[i] = w.b[i] * angle.a[i];
        as[i] = w.a[i] * angle.b[i];
      }
    }
    int h = (k ? s - q_steps : s) * L::kRows + sub;
    __nv_bfloat16 *out = t.out + row * t.out_row + h * t.out_head;
    const long long by = L::kRows * t.out_head;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u >= next) break;
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
      if (h < t.heads) l.store(out, z);
      out += by;
      h += L::kRows;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      x[u][0] = ahead[u][0];
      x[u][1] = ahead[u][1];
    }
  }
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: fills with zeros, reads nothing
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// A warp's steps: a step is 512 bytes of head rows of one row of the batch (the
// queries' steps, then the keys'), and a warp takes a run of them.  They come
// through a ring in shared memory, up to kStages ahead; a row's angles come with
// its first step.
template <int D, bool kPairs>
struct Steps {
  using L = Lane<D, kPairs>;
  static constexpr uint32_t kDz = 512, kAngles = 1024, kStage = 1536;
  static constexpr uint32_t kWarpBytes = kStages * kStage + 16 * ((kStages + 3) / 4);  // and whether they are in the table

  const NormRopeParams &p;
  uint8_t *ring;
  int *ok;
  int lane, sub, q_steps, steps;
  // the place of the next step to be asked for, and of the one at hand
  long long to_ask;
  int ask_row, ask_s, ask_slot = 0, row, s, slot = 0, next_pos;
  bool ask_angles = true, fresh = true;
  const __nv_bfloat16 *x = nullptr, *dz = nullptr;

  __device__ __forceinline__ Steps(const NormRopeParams &p_, uint8_t *smem, int warp, int lane_, long long first,
                                   long long n)
      : p(p_), ring(smem + warp * kWarpBytes), ok(reinterpret_cast<int *>(ring + kStages * kStage)), lane(lane_),
        sub(lane_ / L::kLanes), to_ask(n) {
    q_steps = (p.t[0].heads + L::kRows - 1) / L::kRows;
    steps = q_steps + (p.t[1].heads + L::kRows - 1) / L::kRows;
    ask_row = row = (int)(first / steps);
    ask_s = s = (int)(first - (long long)row * steps);
    if (n > 0) next_pos = p.positions[row];
  }
  __device__ __forceinline__ void ask() {
    if (to_ask > 0) {
      --to_ask;
      const bool k = ask_s >= q_steps;
      const NormRopeTensor &t = p.t[k];
      const int h = (k ? ask_s - q_steps : ask_s) * L::kRows + sub;
      if (ask_angles || ask_s == q_steps) {
        const int c = (lane % L::kLanes) * 8;
        x = t.x + ask_row * t.x_row + h * t.x_head + c;
        dz = t.dz + ask_row * t.dz_row + h * t.dz_head + c;
      }
      const uint32_t at = smem_u32(ring) + ask_slot * kStage;
      const bool real = h < t.heads;  // else the address is not looked at
      cp16(at + lane * 16, x, real);
      cp16(at + kDz + lane * 16, dz, real);
      x += L::kRows * t.x_head;
      dz += L::kRows * t.dz_head;
      if (ask_angles) {
        const int pos = next_pos;
        const bool in = pos >= 0 && pos < p.max_positions;
        if (lane * 4 < p.rot) cp16(at + kAngles + lane * 16, p.rope + (in ? (long long)pos * p.rot + lane * 4 : 0), in);
        if (lane == 0) {
          ok[ask_slot] = in;
          if (!in) atomicCAS(p.status, 0, kStatusBadPosition);
        }
        if (ask_row + 1 < p.rows) next_pos = p.positions[ask_row + 1];
      }
      ask_angles = ++ask_s == steps;
      if (ask_angles) {
        ask_s = 0;
        ++ask_row;
      }
      if (++ask_slot == kStages) ask_slot = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int i = 0; i < kStages - 2; ++i) ask();
  }
  // The next kN steps have come.
  template <int kN>
  __device__ __forceinline__ void take() {
    static_assert(kN <= 2, "two steps more than the ring was filled to");
#pragma unroll
    for (int i = 0; i < kN; ++i) ask();
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
  }
  __device__ __forceinline__ const uint8_t *stage(int i) const {
    const int at = slot + i;
    return ring + (at < kStages ? at : at - kStages) * kStage;
  }
  __device__ __forceinline__ void done(int n) {
    __syncwarp();  // every lane has read the stages
    slot += n;
    if (slot >= kStages) slot -= kStages;
    s += n;
    fresh = s == steps;
    if (fresh) {
      s = 0;
      ++row;
    }
  }
  __device__ __forceinline__ const __nv_bfloat16 *head_row(const uint8_t *stage) const {
    return reinterpret_cast<const __nv_bfloat16 *>(stage) + sub * D;
  }
};

// The steps of warp `w`: p.per_warp each.
__device__ __forceinline__ long long first_step(const NormRopeParams &p, long long w, long long *n) {
  const long long first = w * p.per_warp, left = p.steps - first;
  *n = left < 0 ? 0 : left < p.per_warp ? left : p.per_warp;
  return first;
}

// A warp keeps its sums of dw in registers, the CTA's go to its part.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2) dash_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  using L = Lane<D, kPairs>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  // the sum of the parts may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L::kLanes;
  long long n;
  const long long first = first_step(p, (long long)blockIdx.x * kWarps + warp, &n);
  const L l(lane, p.rot);
  Steps<D, kPairs> steps(p, smem, warp, lane, first, n);
  steps.begin();
  Eight w[2], dw[2], angle;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    w[which] = l.weight(p, which);
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[which].a[i] = dw[which].b[i] = f2(0.f, 0.f);
  }
  F2 minus[2];
  __nv_bfloat16 *out = nullptr;
  // kN steps of the queries or of the keys
  auto step = [&](auto key, auto count) {
    constexpr int which = decltype(key)::value, kN = decltype(count)::value;
    const NormRopeTensor &t = p.t[which];
    steps.template take<kN>();
    const int s = which ? steps.s - steps.q_steps : steps.s, h = s * L::kRows + sub;
    if (steps.fresh) {
      angle = l.angles(reinterpret_cast<const float *>(steps.stage(0) + steps.kAngles), p.rot, steps.ok[steps.slot]);
#pragma unroll
      for (int i = 0; i < 2; ++i) minus[i] = -angle.b[i];
    }
    if (steps.fresh || s == 0) out = t.out + steps.row * t.out_row + h * t.out_head;
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      uint2 xw[2], zw[2];
      l.load(steps.head_row(steps.stage(u)), xw);
      l.load(steps.head_row(steps.stage(u) + steps.kDz), zw);
      const Eight x = L::widen(xw), z = L::widen(zw);
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
      const bool real = h + u * L::kRows < t.heads;
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
      if (real) l.store(out, d);
      out += L::kRows * t.out_head;
    }
    steps.done(kN);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Q = std::integral_constant<int, 0>;
  using K = One;
  while (n > 0) {
    const bool q = steps.s < steps.q_steps, two = n > 1 && steps.s + 2 <= (q ? steps.q_steps : steps.steps);
    if (q) {
      if (two) step(Q(), Two());
      else step(Q(), One());
    } else {
      if (two) step(K(), Two());
      else step(K(), One());
    }
    n -= two ? 2 : 1;
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
  for (int x = threadIdx.x; x < 2 * D; x += kWarps * 32) {
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
constexpr int kSmemBwd = kThreads / 32 * (int)Steps<D, false>::kWarpBytes;

template <int D>
cudaError_t launch_bwd(NormRopeParams &p, cudaStream_t stream) {
  p.steps = norm_steps(p.rows, p.t[0].heads, p.t[1].heads, D);
  const int ctas = norm_bwd_ctas(p.steps);  // 0 without rows: dw is then a sum of nothing
  if (ctas > 0) {
    const long long warps = (long long)ctas * (kThreads / 32);
    p.per_warp = (p.steps + warps - 1) / warps;
    const cudaError_t e = launch(p.pairs ? dash_norm_rope_bwd_kernel<D, true> : dash_norm_rope_bwd_kernel<D, false>,
                                 ctas, kThreads, kSmemBwd<D>, stream, nullptr, p);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr = overlap_attr();
  return launch(dash_norm_rope_sum_kernel, 2 * D / 8, 256, 0, stream, &attr, p, ctas);
}

template <int D>
cudaError_t prepare_t() {
  for (auto kernel : {dash_norm_rope_bwd_kernel<D, true>, dash_norm_rope_bwd_kernel<D, false>})
    if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBwd<D>))
      return e;
  cudaFuncAttributes fa;  // loads the others
  for (auto kernel : {dash_norm_rope_kernel<D, true>, dash_norm_rope_kernel<D, false>})
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
