// The paged key-value cache for sm_103a: attention of one new token per
// sequence, writing new tokens into pages, copying pages.  All three are bound
// by the cache's bytes.
//
// Decode.  Per sequence b and Q head h:
//   x_t = scale log2(e) q.k_t,  m = max x_t,  l = sum 2^(x_t - m),
//   o = (1/l) sum 2^(x_t - m) v_t,  lse = ln2 (m + log2 l).
// A sequence is cut into splits of decode_chunk(length) tokens, a rule on its
// own length alone, so its bits do not depend on the other sequences of the
// batch.  A CTA takes (K/V head, block of 16 Q heads of its group, split); its
// four warps take 16 tokens of every 64 each and run a softmax of their own,
// so nothing but the end of the split synchronises them.  Each warp moves its
// rows with 16-byte asynchronous copies into a ring of its own and feeds them
// to 16 x 8 x 16 matrix instructions, whose 16 rows are the Q heads of the
// group (rows past the group are idle: at 16 flop per cache byte the tensor
// pipe stays far from its limit, while the plain pipe would bound groups of 8).
// P is rounded to bf16 as the product's operand, with l summed from the same
// 32-bit values before the rounding.  A second kernel joins the splits of a
// sequence in their order; calls whose table holds at most one split skip it,
// and in small calls the splits of a sequence are a cluster, which joins them
// through its CTAs' shared memory, with the same bits.
#include <cuda_runtime.h>

#include <atomic>

#include "decode.cuh"
#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

__device__ int g_ops_status;

namespace {
std::atomic<bool> g_ops_used{false};
}
bool ops_status_used() { return g_ops_used.load(); }
cudaError_t ops_status_address(int **p) {
  g_ops_used.store(true);
  return cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_ops_status);
}

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
static_assert(kThreads == kDecodeThreads, "the items are found by all threads");
constexpr int kTok = 16;               // tokens of a warp per step
constexpr int kStep = kWarps * kTok;   // tokens of the CTA per step
constexpr int kStages = 3;

template <int D>
struct DecCfg {
  static constexpr int kRow = D * 2;                         // bytes
  static constexpr int kTile = kTok * kRow;                  // K (or V) rows of a warp's step
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kSmem = kWarps * kWarpBytes;          // the ring; reused to join the warps
  static constexpr int oPart = kWarps * 16 * (D * 4 + 8);    // the split's own result, for its cluster
  static_assert(kSmem >= oPart + 16 * (D * 4 + 8), "the joins fit in the ring");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: fills with zeros, reads nothing
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, Deal kDeal>
__global__ void __launch_bounds__(kThreads, 2) dash_decode_kernel(const DecodeParams p) {
  using C = DecCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the join may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
  const int g = lane >> 2, t4 = lane & 3;

  Items<kDeal> it;
  for (long long item = blockIdx.x;; item += gridDim.x) {
    const int found = it.find(p, item);
    if (found == 0) break;
    if (found < 0) continue;
    const int b = it.b, split = it.split, rest = it.rest;
    const int hk = rest / p.hblocks, hb = rest - hk * p.hblocks;
    const int h0 = hk * p.group + hb * 16, nh = min(16, p.group - hb * 16);
    const int len = decode_len(p, b);
    const int chunk = decode_chunk(len, p.least_chunk), n_splits = max(1, decode_splits(len, p.least_chunk));
    const bool mine = kDeal != kCluster || split < n_splits;  // or the sequence does not have this split of the cluster
    const int begin = split * chunk, end = min(len, begin + chunk);
    const int steps = mine ? (end - begin + kStep - 1) / kStep : 0;
    const int *table = p.table + b * p.table_row;

    // Q fragments: rows g and g + 8 of the block's 16 heads
    uint32_t qf[D / 16][4];
    {
      const __nv_bfloat16 *q = p.q + b * p.q_batch + h0 * p.q_head;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = g + (i & 1) * 8, col = 16 * kk + 2 * t4 + (i >> 1) * 8;
          qf[kk][i] = row < nh ? *reinterpret_cast<const uint32_t *>(q + row * p.q_head + col) : 0u;
        }
    }

    // A lane below 16 keeps the row of one of the warp's tokens.
    auto page_of = [&](int step) -> int {
      const int t = begin + step * kStep + warp * kTok + (lane & 15);
      return t < end ? (t < p.shared ? p.table : table)[(p.first + t) / p.page_size] : -1;
    };
    uint32_t valid_ring[kStages];  // the tokens of each stage that count
    auto load = [&](int step, int page, int slot) -> uint32_t {
      const int t = begin + step * kStep + warp * kTok + (lane & 15);
      const bool inside = step < steps && t < end;
      const bool ok = inside && page >= 0 && page < p.n_pages;
      if (inside && !ok) atomicCAS(p.status, 0, kStatusBadPage);
      const int off = (p.first + t) % p.page_size;
      const long long pg = ok ? page : 0;
      const long long ka = ok ? pg * p.ks.page + off * p.ks.token + hk * p.ks.head : 0;
      const long long va = ok ? pg * p.vs.page + off * p.vs.token + hk * p.vs.head : 0;
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;
      const uint32_t dst = ring + slot * C::kStage;
      const int c = lane % kChunks, rsub = lane / kChunks;
      if (step < steps) {
#pragma unroll
        for (int i = 0; i < kTok / kRowsPer; ++i) {
          const int r = i * kRowsPer + rsub;
          const long long kr = __shfl_sync(0xffffffffu, ka, r), vr = __shfl_sync(0xffffffffu, va, r);
          const bool v = (valid >> r) & 1u;
          const uint32_t at = dst + r * C::kRow + ((c ^ (r & 7)) << 4);
          cp16(at, p.k + kr + c * 8, v);
          cp16(at + C::kTile, p.v + vr + c * 8, v);
        }
      }
      cp_commit();
      return valid;
    };

    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int page = page_of(0);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      const int nxt = page_of(s + 1);
      valid_ring[s] = load(s, page, s);
      page = nxt;
    }
    for (int step0 = 0; step0 < steps; step0 += kStages) {
#pragma unroll
      for (int slot = 0; slot < kStages; ++slot) {
        const int step = step0 + slot;
        if (step >= steps) break;
        constexpr int kAhead = kStages - 1;
        const int nslot = (slot + kAhead) % kStages;
        __syncwarp();  // the slot to be refilled has been read by every lane
        const int nxt = page_of(step + kAhead + 1);
        valid_ring[nslot] = load(step + kAhead, page, nslot);
        page = nxt;
        cp_wait<kAhead>();
        __syncwarp();
        const uint32_t kb = ring + slot * C::kStage, vb = kb + C::kTile;
        // S = Q K^T: 16 heads x 16 tokens
        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t r[4];
          const int row = (lane & 7) + ((lane >> 4) << 3), c = 2 * kk + ((lane >> 3) & 1);
          ldsm4(kb + row * C::kRow + ((c ^ (row & 7)) << 4), r);
          mma16816(s[0], qf[kk], r[0], r[1]);
          mma16816(s[1], qf[kk], r[2], r[3]);
        }
        const uint32_t valid = valid_ring[slot];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 8 * n + 2 * t4 + (i & 1);
            s[n][i] = ((valid >> t) & 1u) ? s[n][i] * p.scale_log2 : -INFINITY;
          }
        uint32_t pf[4];
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float m_new = fmaxf(m[r], top);
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing counted yet
          f[r] = ex2(m[r] - ref);
          m[r] = m_new;
          const float a0 = ex2(s[0][2 * r] - ref), a1 = ex2(s[0][2 * r + 1] - ref);
          const float a2 = ex2(s[1][2 * r] - ref), a3 = ex2(s[1][2 * r + 1] - ref);
          l[r] = l[r] * f[r] + ((a0 + a1) + (a2 + a3));
          pf[r] = pack_bf16(a0, a1);
          pf[2 + r] = pack_bf16(a2, a3);
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            acc[n][0] *= f[0];
            acc[n][1] *= f[0];
            acc[n][2] *= f[1];
            acc[n][3] *= f[1];
          }
        }
        // O += P V
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t r[4];
          const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c = 2 * n + (lane >> 4);
          ldsm4t(vb + row * C::kRow + ((c ^ (row & 7)) << 4), r);
          mma16816(acc[2 * n], pf, r[0], r[1]);
          mma16816(acc[2 * n + 1], pf, r[2], r[3]);
        }
      }
    }
    cp_wait<0>();
    // ---- join the four warps: each scales to the split's maximum
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();  // every warp has left its ring
    float *s_o = reinterpret_cast<float *>(smem);                        // [warp][16][D]
    float2 *s_ml = reinterpret_cast<float2 *>(smem + kWarps * 16 * D * 4);  // [warp][16]
    if (t4 == 0) {
      s_ml[warp * 16 + g] = make_float2(m[0], l[0]);
      s_ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      // columns are rotated by the row so that the rows of a store do not share banks
      const int c = 8 * n + 2 * t4;
      float *o0 = s_o + (warp * 16 + g) * D, *o1 = o0 + 8 * D;
      *reinterpret_cast<float2 *>(o0 + ((c + 8 * g) & (D - 1))) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2 *>(o1 + ((c + 8 * g) & (D - 1))) = make_float2(acc[n][2], acc[n][3]);
    }
    __syncthreads();
    constexpr int kVec = D / 4;  // float4 per row
    for (int x = threadIdx.x; mine && x < nh * kVec; x += kThreads) {
      const int row = x / kVec, c = (x - row * kVec) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w * 16 + row].x);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * 16 + row];
        const float fw = ex2(ml.x - ref);
        ll += fw * ml.y;
        const float4 v = *reinterpret_cast<const float4 *>(s_o + (w * 16 + row) * D + ((c + 8 * (row & 7)) & (D - 1)));
        o[0] += fw * v.x;
        o[1] += fw * v.y;
        o[2] += fw * v.z;
        o[3] += fw * v.w;
      }
      const float inv = inverse_sum(ll);
      const int h = h0 + row;
      if (p.parts_before + n_splits == 1) {
        uint2 w;
        w.x = pack_bf16(o[0] * inv, o[1] * inv);
        w.y = pack_bf16(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2 *>(p.o + b * p.o_batch + h * p.o_head + c) = w;
        if (c == 0 && p.lse) p.lse[(size_t)b * p.Hq + h] = log_sum(mm, ll);
      } else if (kDeal == kCluster) {
        float *part = reinterpret_cast<float *>(smem + C::oPart);  // [16][D], then [16] {maximum, sum}
        *reinterpret_cast<float4 *>(part + row * D + c) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        if (c == 0) reinterpret_cast<float2 *>(part + 16 * D)[row] = make_float2(mm, ll);
      } else {
        const size_t at = ((size_t)b * p.Hq + h) * (p.parts_before + p.max_splits) + p.parts_before + split;
        *reinterpret_cast<float4 *>(p.part_o + at * D + c) =
            make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        if (c == 0) p.part_ml[at] = make_float2(mm, ll);
      }
    }
    if (kDeal == kCluster) {
      if (n_splits > 1) {  // the same in every CTA of the cluster
        join_cluster<D>(p, smem + C::oPart, b, h0, nh, split, n_splits);
      }
      break;
    }
    __syncthreads();  // the ring is free for the next item
  }
  // where this grid was let in before the end of the prefix's, its own end says that both have ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One Q head's attention of the first `len` tokens, which lie in the pages of the
// table's first row: a block of 128 threads takes 128 tokens at a time, a thread
// a score and then a value of the row.  What does not count is not multiplied.
template <int D>
__device__ __noinline__ void attend_row(const DecodeParams &p, int b, int h, int len, float *s_w, int *s_page,
                                        float *s_m) {
  const int tid = threadIdx.x, hk = h / p.group;
  const __nv_bfloat16 *q = p.q + b * p.q_batch + h * p.q_head;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int t0 = 0; t0 < len; t0 += 128) {
    const int t = t0 + tid, page = t < len ? p.table[t / p.page_size] : -1;
    const bool ok = page >= 0 && page < p.n_pages;
    float x = -INFINITY;
    if (ok) {
      const __nv_bfloat16 *k = p.k + page * p.ks.page + t % p.page_size * p.ks.token + hk * p.ks.head;
      float dot = 0.f;
      for (int c = 0; c < D; c += 8) {
        const uint4 kw = *reinterpret_cast<const uint4 *>(k + c), qw = *reinterpret_cast<const uint4 *>(q + c);
        const uint32_t a[4] = {kw.x, kw.y, kw.z, kw.w}, e[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(e[i] << 16), dot);
          dot = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(e[i] & 0xffff0000u), dot);
        }
      }
      x = dot * p.scale_log2;
    }
    float top = x;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    if ((tid & 31) == 0) s_m[tid >> 5] = top;
    __syncthreads();
    const float m1 = fmaxf(m, fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])));
    const float ref = m1 == -INFINITY ? 0.f : m1, f = ex2(m - ref);
    m = m1;
    l *= f;
    o *= f;
    s_w[tid] = ex2(x - ref);
    s_page[tid] = ok ? page : -1;
    __syncthreads();
    for (int i = 0; i < 128; ++i) {
      if (s_page[i] < 0) continue;
      l += s_w[i];
      if (tid < D)
        o = fmaf(s_w[i], __bfloat162float(p.v[s_page[i] * p.vs.page + (t0 + i) % p.page_size * p.vs.token +
                                              hk * p.vs.head + tid]), o);
    }
    __syncthreads();
  }
  if (tid < D) p.o[b * p.o_batch + h * p.o_head + tid] = __float2bfloat16_rn(o * inverse_sum(l));
  if (tid == 0 && p.lse) p.lse[(size_t)b * p.Hq + h] = log_sum(m, l);
}

// Joins the splits of a (sequence, Q head) in their order.  kPrefix: parts of a
// shared prefix are among them.  Its products take a token that one sequence
// attends and a shorter one does not with a weight of 0 for the latter, and 0 times
// a NaN or an infinity in that token's V is a NaN.  So where a sequence ends inside
// the prefix and its row is not finite, the row is made anew from the tokens that it
// has: the masked ones are then the cause, or the row is not finite by its own.
template <int D, bool kPrefix>
__global__ void __launch_bounds__(128) dash_decode_join(const DecodeParams p) {
  // every block waits, so that this grid never ends before the first one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = p.parts_before + decode_splits(decode_len(p, b), p.least_chunk);
  if (n <= 1 && p.parts_before == 0) return;  // written by the first kernel
  const size_t at = ((size_t)b * p.Hq + h) * (p.parts_before + p.max_splits);
  __shared__ __align__(16) float s_w[128];
  __shared__ float s_m[4];
  __shared__ float4 s_o[128];
  using J = Join<D>;
  const int tid = threadIdx.x, c = tid % J::kVec, part = tid / J::kVec;
  // the first rows are on their way while the weights are made
  constexpr int kAhead = 8;
  const float *row = p.part_o + at * D + 4 * c;
  float4 v[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = part + k * J::kPart;
    v[k] = i < n ? *reinterpret_cast<const float4 *>(row + (size_t)i * D) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // at most 128 splits: one per thread
  const float2 ml = tid < n ? p.part_ml[at + tid] : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) s_m[tid >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float ref = m == -INFINITY ? 0.f : m;
  s_w[tid] = J::weight(ml, ref);
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (part + k * J::kPart < n) J::add(o, s_w[part + k * J::kPart], v[k]);
#pragma unroll 8
  for (int i = part + kAhead * J::kPart; i < n; i += J::kPart)
    J::add(o, s_w[i], *reinterpret_cast<const float4 *>(row + (size_t)i * D));
  if (kPrefix) {
    const int len = max(0, min(p.lengths[b], p.max_pages * p.page_size));
    // a part that weighs 0 counts too: 0 times what is not finite is a NaN
    if (len < p.first && __syncthreads_or(!isfinite(o.x) || !isfinite(o.y) || !isfinite(o.z) || !isfinite(o.w))) {
      attend_row<D>(p, b, h, len, s_w, reinterpret_cast<int *>(s_o), s_m);
      return;
    }
  }
  s_o[tid] = o;
  // the weights' sum, in their order (those behind the last split are 0)
  float l = 0.f;
  for (int i = 0; i < n; i += 4) {
    const float4 w = *reinterpret_cast<const float4 *>(s_w + i);
    l = ((l + w.x) + w.y) + w.z;
    l += w.w;
  }
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int k = 1; k < J::kPart; ++k) {
      const float4 u = s_o[k * J::kVec + c];
      o = make_float4(o.x + u.x, o.y + u.y, o.z + u.z, o.w + u.w);
    }
    J::write(p, b, h, 4 * c, o, m, l);
  }
}

template <int D>
cudaError_t launch_decode_t(const DecodeParams &p, int num_sms, cudaStream_t stream) {
  using C = DecCfg<D>;
  const long long items = (long long)p.B * p.max_splits * p.Hkv * p.hblocks;
  if (p.parts_before == 0 && decode_clustered(p.B, p.Hq, p.max_splits)) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.max_splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    return launch(dash_decode_kernel<D, kCluster>, (int)items, kThreads, C::kSmem, stream, &attr, p);
  }
  // Two CTAs fit on an SM.  Where they hold every item that the table has room
  // for, the scan is left out (one sequence of 701 tokens on 4 K/V heads, before
  // it was a cluster's: 6.3 us against 7.0).
  const bool all = items <= 2LL * num_sms;
  cudaLaunchAttribute attr = overlap_attr();
  const cudaError_t e = launch(all ? dash_decode_kernel<D, kPlain> : dash_decode_kernel<D, kScan>,
                               all ? (int)items : 2 * num_sms, kThreads, C::kSmem, stream,
                               p.parts_before > 0 ? &attr : nullptr, p);
  return e != cudaSuccess || p.parts_before + p.max_splits <= 1 ? e : launch_decode_join(D, p, stream);
}

// ------------------------------------------------------------------ write
// A warp takes a token: its K and V rows of all heads, 16 bytes a lane.
__global__ void __launch_bounds__(256) dash_cache_write_kernel(const CacheWriteParams p) {
  const int lane = threadIdx.x & 31;
  const int nwarps = gridDim.x * 8;
  const int vecs = p.D >> 3, total = p.heads * vecs;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < p.n_tokens; t += nwarps) {
    // the sequence of the token: the last b with cu[b] <= t
    int lo = 0, hi = p.B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid + 1] <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo >= p.B) continue;  // rows behind the last sequence
    const int b = lo, first = p.cu[b];
    const long long pos = (long long)p.starts[b] + (t - first);
    const long long slot = pos / p.page_size;
    int page = -1;
    if (t >= first && pos >= 0 && slot < p.max_pages) page = p.table[b * p.table_row + slot];
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) atomicCAS(p.status, 0, kStatusBadPage);
      continue;
    }
    const int off = (int)(pos - slot * p.page_size);
    const __nv_bfloat16 *k = p.k + t * p.k_row, *v = p.v + t * p.v_row;
    __nv_bfloat16 *kp = p.kp + page * p.ks.page + off * p.ks.token;
    __nv_bfloat16 *vp = p.vp + page * p.vs.page + off * p.vs.token;
    constexpr int kU = 4;
    for (int x0 = lane; x0 < total; x0 += 32 * kU) {
      uint4 a[kU], c[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int x = x0 + 32 * u;
        if (x < total) {
          const int h = x / vecs, e = (x - h * vecs) * 8;
          a[u] = *reinterpret_cast<const uint4 *>(k + h * p.k_head + e);
          c[u] = *reinterpret_cast<const uint4 *>(v + h * p.v_head + e);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int x = x0 + 32 * u;
        if (x < total) {
          const int h = x / vecs, e = (x - h * vecs) * 8;
          *reinterpret_cast<uint4 *>(kp + h * p.ks.head + e) = a[u];
          *reinterpret_cast<uint4 *>(vp + h * p.vs.head + e) = c[u];
        }
      }
    }
  }
}

// ------------------------------------------------------------------- copy
// The pairs travel in the launch's arguments: nothing on the device holds
// them, so a captured call keeps its own and two calls share nothing.
template <int N>
struct PairList {
  int2 p[N];
};

// Work is (pair, K or V, piece of the page); a page's tokens and heads are
// walked 16 bytes a thread, kU of them in flight.
template <int N>
__global__ void __launch_bounds__(256)
    dash_cache_copy_kernel(const __grid_constant__ PairList<N> pairs, const CacheCopyParams p, int pieces) {
  const int vecs = p.D >> 3;
  const int total = p.page_size * p.heads * vecs;  // 16-byte vectors of a page
  const int pair = blockIdx.x / pieces, piece = blockIdx.x - pair * pieces;
  const int2 pr = pairs.p[pair];
  const bool is_v = blockIdx.y != 0;
  __nv_bfloat16 *base = is_v ? p.vp : p.kp;
  const CacheStrides st = is_v ? p.vs : p.ks;
  const __nv_bfloat16 *src = base + pr.x * st.page;
  __nv_bfloat16 *dst = base + pr.y * st.page;
  constexpr int kU = 8;
  // the page is one run of bytes
  const bool flat = (st.head == p.D || p.heads == 1) && (st.token == (long long)p.heads * p.D || p.page_size == 1);
  for (int x0 = piece * 256 * kU + threadIdx.x; x0 < total; x0 += pieces * 256 * kU) {
    uint4 a[kU];
    long long at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = x0 + 256 * u;
      if (x < total) {
        if (flat) {
          at[u] = (long long)x * 8;
        } else {
          const int row = x / vecs, tok = row / p.heads;
          at[u] = tok * st.token + (row - tok * p.heads) * st.head + (x - row * vecs) * 8;
        }
        a[u] = *reinterpret_cast<const uint4 *>(src + at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (x0 + 256 * u < total) *reinterpret_cast<uint4 *>(dst + at[u]) = a[u];
  }
}

template <int N>
cudaError_t launch_copy_t(const CacheCopyParams &p, const int2 *pairs, int n, cudaStream_t stream) {
  PairList<N> list;
  for (int i = 0; i < n; ++i) list.p[i] = pairs[i];
  const long long total = (long long)p.page_size * p.heads * (p.D / 8);
  const int pieces = (int)((total + 2047) / 2048 < 64 ? (total + 2047) / 2048 : 64);
  return launch(dash_cache_copy_kernel<N>, dim3(n * pieces, 2), 256, 0, stream, nullptr, list, p, pieces);
}

}  // namespace

template <int D>
static cudaError_t prepare_decode_t() {
  cudaError_t e = cudaSuccess;
  for (auto kernel : {dash_decode_kernel<D, kPlain>, dash_decode_kernel<D, kScan>, dash_decode_kernel<D, kCluster>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<D>::kSmem);
  return e;
}
cudaError_t prepare_decode() {
  const cudaError_t e = prepare_decode_t<64>();
  return e != cudaSuccess ? e : prepare_decode_t<128>();
}

cudaError_t launch_decode_join(int D, const DecodeParams &p, cudaStream_t stream) {
  cudaLaunchAttribute attr = overlap_attr();
  auto *kernel = p.parts_before > 0 ? (D == 64 ? dash_decode_join<64, true> : dash_decode_join<128, true>)
                                    : (D == 64 ? dash_decode_join<64, false> : dash_decode_join<128, false>);
  return launch(kernel, dim3(p.Hq, p.B), 128, 0, stream, &attr, p);
}

cudaError_t launch_decode(int D, const DecodeParams &p, int num_sms, cudaStream_t stream) {
  return D == 64 ? launch_decode_t<64>(p, num_sms, stream) : launch_decode_t<128>(p, num_sms, stream);
}

cudaError_t launch_cache_write(const CacheWriteParams &p, int num_sms, cudaStream_t stream) {
  const int want = (p.n_tokens + 7) / 8;
  return launch(dash_cache_write_kernel, want < 8 * num_sms ? want : 8 * num_sms, 256, 0, stream, nullptr, p);
}

cudaError_t launch_cache_copy(const CacheCopyParams &p, const int2 *pairs, int n, cudaStream_t stream) {
  for (int i = 0; i < n; i += kCopyPairs) {
    const int k = n - i < kCopyPairs ? n - i : kCopyPairs;
    const cudaError_t e =
        k <= 64 ? launch_copy_t<64>(p, pairs + i, k, stream) : launch_copy_t<kCopyPairs>(p, pairs + i, k, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dash
