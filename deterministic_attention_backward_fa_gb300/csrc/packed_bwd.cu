// Preprocess and convert of the packed backward; its main kernel is
// dash_bwd_main (bwd.cu) with kPacked.
//
// Both are bound by the bytes they move.  A block takes one (tile, Q head), so
// a packed row is found without a search, and rows past a sequence's end get
// lse2 = +inf (P = 0) and delta = 0 in the padded row arrays.
#include <cuda_runtime.h>

#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

// A copy of `src` bounded to one sequence: rows past its end lie outside the
// map, so the copies fill them with zeros instead of another sequence's rows
// (whose values, times P = 0, could still be NaN).
__device__ __forceinline__ void bound_map(CUtensorMap *dst, const CUtensorMap *src, const void *base, int rows) {
  const int4 *s = reinterpret_cast<const int4 *>(src);
  int4 *d = reinterpret_cast<int4 *>(dst);
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = s[i];
  const uint64_t at = reinterpret_cast<uint64_t>(dst);
  asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(at),
               "l"(reinterpret_cast<uint64_t>(base))
               : "memory");
  asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(at), "r"(rows) : "memory");
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(256)
    dash_packed_preprocess(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                           const PackedPreParams p) {
  const int gt = blockIdx.x, h = blockIdx.y;
  const int4 tile = p.tiles[gt];  // {first row inside the sequence, valid rows, sequence, first packed row}
  if (h == 0 && tile.x == 0 && threadIdx.x < 4) {
    const int2 sq = p.seqs[tile.z];
    const CUtensorMap *src = threadIdx.x == 0 ? &tmQ : threadIdx.x == 1 ? &tmK : threadIdx.x == 2 ? &tmV : &tmDO;
    bound_map(p.maps + 4 * (size_t)tile.z + threadIdx.x, src,
              static_cast<const uint8_t *>(p.base[threadIdx.x]) + sq.x * p.base_row[threadIdx.x], sq.y);
  }
  const size_t key = (size_t)h * p.n_tiles + gt;
  if (threadIdx.x < kSemStride) p.sem[key * kSemStride + threadIdx.x] = 0;
  // D / 8 lanes of 16 bytes per row; every thread has all its loads in flight at once
  constexpr int kLanesPerRow = D / 8, kRowsPerPass = 256 / kLanesPerRow, kPasses = kPackedTile / kRowsPerPass;
  const int r0 = threadIdx.x / kLanesPerRow, li = threadIdx.x % kLanesPerRow;
  const __nv_bfloat16 *o = p.o + tile.w * p.o_row + h * p.o_head + li * 8;
  const __nv_bfloat16 *g = p.dout + tile.w * p.do_row + h * p.do_head + li * 8;
  uint4 a[kPasses], b[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int r = r0 + u * kRowsPerPass;
    a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
    if (r < tile.y) {
      a[u] = *reinterpret_cast<const uint4 *>(o + r * p.o_row);
      b[u] = *reinterpret_cast<const uint4 *>(g + r * p.do_row);
    }
  }
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int r = r0 + u * kRowsPerPass;
    const __nv_bfloat162 *pa = reinterpret_cast<const __nv_bfloat162 *>(&a[u]);
    const __nv_bfloat162 *pb = reinterpret_cast<const __nv_bfloat162 *>(&b[u]);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 fa = __bfloat1622float2(pa[i]), fb = __bfloat1622float2(pb[i]);
      sum = fmaf(fa.x, fb.x, sum);
      sum = fmaf(fa.y, fb.y, sum);
    }
#pragma unroll
    for (int off = kLanesPerRow / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (li == 0) {
      const bool valid = r < tile.y;
      p.delta[key * kPackedTile + r] = sum;
      p.lse2[key * kPackedTile + r] =
          valid ? p.lse[h * p.lse_head + tile.w + r] * 1.4426950408889634f : __int_as_float(0x7f800000);
    }
  }
}

// dQ = bf16(scale * accumulator): the only rounding of dQ below 32 bits.
template <int D>
__global__ void __launch_bounds__(256) dash_packed_convert(const PackedConvertParams p) {
  const int gt = blockIdx.x, h = blockIdx.y;
  const int4 tile = p.tiles[gt];
  const float *acc = p.accum + ((size_t)h * p.n_tiles + gt) * (size_t)(kPackedTile * D);
  constexpr int kGroups = D / 16;  // a thread turns 16 columns of a row into 32 bytes
#pragma unroll
  for (int i = threadIdx.x; i < kPackedTile * kGroups; i += 256) {
    const int r = i & (kPackedTile - 1), gidx = i >> 7;
    if (r >= tile.y) continue;
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = *reinterpret_cast<const float4 *>(acc + ((size_t)(4 * gidx + k) * kPackedTile + r) * 4);
    uint4 o[2];
    uint32_t *w = reinterpret_cast<uint32_t *>(o);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[2 * k] = pack_bf16(p.scale * v[k].x, p.scale * v[k].y);
      w[2 * k + 1] = pack_bf16(p.scale * v[k].z, p.scale * v[k].w);
    }
    uint4 *out = reinterpret_cast<uint4 *>(p.dq + (long long)(tile.w + r) * p.dq_row + h * p.dq_head + 16 * gidx);
    out[0] = o[0];
    out[1] = o[1];
  }
}

}  // namespace

cudaError_t launch_packed_preprocess(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                     const CUtensorMap &dout, const PackedPreParams &p, cudaStream_t stream) {
  const dim3 grid(p.n_tiles, p.heads);
  if (D == 64)
    dash_packed_preprocess<64><<<grid, 256, 0, stream>>>(q, k, v, dout, p);
  else
    dash_packed_preprocess<128><<<grid, 256, 0, stream>>>(q, k, v, dout, p);
  return cudaGetLastError();
}

cudaError_t launch_packed_convert(int D, const PackedConvertParams &p, cudaStream_t stream) {
  const dim3 grid(p.n_tiles, p.heads);
  if (D == 64)
    dash_packed_convert<64><<<grid, 256, 0, stream>>>(p);
  else
    dash_packed_convert<128><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dash
