// What the decode kernels share (paged.cu, cache8.cu): how a CTA finds its
// items, and how the splits of a sequence are joined.
#pragma once

#include <cuda_runtime.h>

#include "packed.h"
#include "sm103.cuh"

namespace dash {

constexpr int kDecodeThreads = 128;

namespace dev {

// How a CTA finds its items.
enum Deal {
  kPlain,    // every sequence has max_splits numbers, those it does not need return at once
  kScan,     // only the splits that a sequence has are numbered
  kCluster,  // as kPlain, and the splits are a cluster
};

// A row's 1 / l and LSE.  l is 0 for a row that attends nothing (o = 0, LSE =
// -inf) and NaN where a score is NaN or +inf: the row's results are then NaN, as
// softmax makes them.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The join of a sequence's splits, in one order whoever makes it: weights
// l 2^(m - max), their sum over the splits in turn, and the weighted rows in
// kPart sums of every kPart-th split, added in turn.  A split that attends
// nothing weighs 0 (m = -inf, l = 0) and its row is 0; nothing is left out by a
// comparison, which would lose a split whose l is NaN.
template <int D>
struct Join {
  static constexpr int kVec = D / 4, kPart = 128 / kVec;  // float4 of a row, sums
  static __device__ __forceinline__ float weight(float2 ml, float ref) { return ml.y * ex2(ml.x - ref); }
  static __device__ __forceinline__ void add(float4 &o, float w, float4 v) {
    o = make_float4(fmaf(w, v.x, o.x), fmaf(w, v.y, o.y), fmaf(w, v.z, o.z), fmaf(w, v.w, o.w));
  }
  static __device__ __forceinline__ void write(const DecodeParams &p, int b, int h, int c, float4 o, float m, float l) {
    const float inv = inverse_sum(l);
    uint2 w;
    w.x = pack_bf16(o.x * inv, o.y * inv);
    w.y = pack_bf16(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(p.o + b * p.o_batch + h * p.o_head + c) = w;
    if (c == 0 && p.lse) p.lse[(size_t)b * p.Hq + h] = log_sum(m, l);
  }
};

// Loads from the shared memory of any CTA of the cluster.
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Joins the splits of a sequence, which are the CTAs of a cluster: every CTA has
// its `nh` rows as fp32 [16][D], then {maximum, sum} [16], at the same `part` of
// its shared memory.
template <int D>
__device__ __forceinline__ void join_cluster(const DecodeParams &p, const uint8_t *smem_part, int b, int h0, int nh,
                                             int split, int n_splits) {
  using J = Join<D>;
  constexpr int kVec = D / 4;
  __syncwarp();
  cluster_sync_all();
  const float *part = reinterpret_cast<const float *>(smem_part);
  const float2 *mls = reinterpret_cast<const float2 *>(part + 16 * D);
  for (int x = split * kDecodeThreads + threadIdx.x; x < nh * kVec; x += p.max_splits * kDecodeThreads) {
    const int row = x / kVec, c = (x - row * kVec) * 4;
    float2 ml[kMaxCluster];
    float4 v[kMaxCluster];
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i < n_splits) {
        ml[i] = ld_cluster2(mapa_rank(mls + row, i));
        v[i] = ld_cluster4(mapa_rank(part + row * D + c, i));
      }
    }
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) m = fmaxf(m, ml[i].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float4 o[J::kPart] = {};
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i)
      if (i < n_splits) {
        const float w = J::weight(ml[i], ref);
        l += w;
        J::add(o[i % J::kPart], w, v[i]);
      }
#pragma unroll
    for (int k = 1; k < J::kPart; ++k)
      o[0] = make_float4(o[0].x + o[k].x, o[0].y + o[k].y, o[0].z + o[k].z, o[0].w + o[k].w);
    J::write(p, b, h0 + row, c, o[0], m, l);
  }
  __syncwarp();
  cluster_sync_all();  // nobody leaves while its results are read
}

// The tokens of sequence b that the decode kernels attend: those behind p.first.
__device__ __forceinline__ int decode_len(const DecodeParams &p, int b) {
  return max(0, min(p.lengths[b], p.max_pages * p.page_size) - p.first);
}

// Items are numbered (sequence, split, K/V head, block of Q heads), the split
// last in clusters.  With kScan the item's sequence is found by scanning the
// splits of kDecodeThreads sequences at a time; `base` and `base_b` remember the
// block of sequences reached so far.  All threads of the CTA ask together.
template <Deal kDeal>
struct Items {
  long long base = 0;  // splits before sequence base_b
  int base_b = 0, in_block = -1;
  int b, split, rest;  // what find() found

  // 1: found, 0: there is no such item and none behind it, -1: its sequence does not have that split
  __device__ __forceinline__ int find(const DecodeParams &p, long long item) {
    __shared__ int s_prefix[kDecodeThreads + 1];
    __shared__ int s_find[2];  // {sequence, splits before it}
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_split = p.Hkv * p.hblocks;
    const long long want = item / per_split;
    b = -1, split = 0, rest = (int)(item - want * per_split);
    if (kDeal == kCluster) {
      if (item >= (long long)p.B * p.max_splits * per_split) return 0;
      const int group = (int)(item / p.max_splits);
      b = group / per_split;
      rest = group - b * per_split;
      split = (int)item - group * p.max_splits;
    } else if (kDeal == kPlain) {
      if (want >= (long long)p.B * p.max_splits) return 0;
      b = (int)(want / p.max_splits);
      split = (int)(want - (long long)b * p.max_splits);
      if (split > 0 && split >= decode_splits(decode_len(p, b), p.least_chunk)) return -1;
    }
    while (kDeal == kScan) {
      if (in_block != base_b) {  // the block's prefix sums
        __syncthreads();
        const int mine = base_b + (int)threadIdx.x;
        int n = 0;
        if (mine < p.B) n = decode_splits(decode_len(p, mine), p.least_chunk);
        // an empty sequence still has an item, which writes its zero row
        if (mine < p.B && n == 0) n = 1;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        s_prefix[threadIdx.x + 1] = x;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += s_prefix[(w + 1) * 32];
        __syncthreads();
        s_prefix[threadIdx.x + 1] = x + before;
        if (threadIdx.x == 0) s_prefix[0] = 0;
        __syncthreads();
        in_block = base_b;
      }
      const int total = s_prefix[kDecodeThreads];
      if (want < base + total) {
        const int off = (int)(want - base);
        if (off >= s_prefix[threadIdx.x] && off < s_prefix[threadIdx.x + 1]) {
          s_find[0] = base_b + threadIdx.x;
          s_find[1] = off - s_prefix[threadIdx.x];
        }
        __syncthreads();
        b = s_find[0];
        split = s_find[1];
        break;
      }
      if (base_b + kDecodeThreads >= p.B) break;
      base += total;
      base_b += kDecodeThreads;
    }
    return b < 0 ? 0 : 1;
  }
};

}  // namespace dev
}  // namespace dash
