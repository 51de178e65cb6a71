// The 8-bit paged key-value cache for sm_103a: writing and reading rows, copying
// pages, attention of one new token per sequence.  All are bound by bytes.
//
// A row (one token of one K/V head) is D codes in e4m3 and a scale, its values
// code x scale.  The scale is the smallest power of two (2^-126 at least) with
// |x| <= 448 scale for the whole row, so that x / scale is exact and each value
// is rounded once, to the nearest code (ties to even); and a row read back in
// bf16 is exact.  (With floating-point codes a finer scale gains nothing: the
// step of a value goes with the value's own power of two.)  A row that holds a
// NaN or an infinity gets a NaN as its scale, and reads as NaN.
//
// Decode.  As in paged.cu, with the rows' scales a_t of K and c_t of V:
//   x_t = scale log2(e) a_t (q . k_t),  o = (1/l) sum 2^(x_t - m) c_t v_t.
// The codes are widened to f16, which holds them exactly, and multiplied there:
//   S^T [16 tokens x 8 heads] = K Q^T,   O^T [16 dims x 8 heads] += V^T P^T
// so that the codes are the large operand and the 8 columns are the heads of a
// group.  Contraction order is free, so a lane takes what lies side by side: of K
// the 16 bytes at 16 (lane % 4) of two tokens, of V the same D / 8 dims of four;
// what it multiplies, it has fetched itself, and its asynchronous copies need
// shared memory only as a queue of its own: no swizzle, no ldmatrix, no exchange.
// Q is multiplied by a power of two first (its largest value lands at 2^14), so
// that f16 holds its 8 bits down to 2^-29 of that.
// P goes to f16 as 2^(x_t - M) c_t with M the maximum of x_t + log2 c_t of its
// head, not of x_t: what counts in O keeps f16's 11 bits whatever the scales
// of V are, and a weight of less than 2^-25 of the largest, which f16 gives up, is
// 2^-11 of it even 16384 times, the longest split of a warp's four.  l and O are 32-bit sums, l of the unrounded 2^(x_t - m).
// m and M move only when a term has grown past 2^8 of them (most steps need no
// reduction across lanes and no rescaling).
// This form takes calls whose items all run at once or are short (701 tokens, 16 heads on 4:
// 7.2 us, a chain of length, page, rows, products and the cluster's join) and
// groups of 9 to 16 heads (64 sequences of 8192 tokens, 16 heads on 1 of 128: 61
// us, 2.3 TB/s, bound by latency: two tiles of heads take 241 registers, so that 8
// warps of an SM stand in each step's chain of copies, widening, scores and weights
// and issue in 30 % of their cycles); decode8.cu has the one for calls that fill the
// GPU.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache8.h"
#include "decode.cuh"
#include "fp8.cuh"
#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

// ------------------------------------------------------------------ codes
// The scale's exponent field for a row whose largest magnitude has the bf16 bits
// `top` (below 0x7f80): 448 = 1.75 x 2^8, so a mantissa of up to 0x60 fits with
// 8 less, and one above it needs 7 less.
__device__ __forceinline__ int scale_field(uint32_t top) {
  return max(1, (int)(top >> 7) - 8 + ((top & 0x7fu) > 0x60u));
}

// ---------------------------------------------------------- write and read
// Where token t of the call lies: its page and place, or -1.  All lanes ask
// together; the sequence (the last b with cu[b] <= t) is found 32 ways at a time,
// since each look-up waits for the one before.
struct Place {
  int page, off;
  bool behind;  // the token is behind the last sequence
};
__device__ __forceinline__ Place place_of(const Cache8RowsParams &p, int t, int lane) {
  int lo = 0, n = p.B;
  while (n > 32) {
    const int step = (n + 31) >> 5, at = (lane + 1) * step;
    const int whole = __popc(__ballot_sync(0xffffffffu, at <= n && p.cu[lo + at] <= t));
    lo += whole * step;
    n = min(step, n - whole * step);
  }
  lo += __popc(__ballot_sync(0xffffffffu, lane < n && p.cu[lo + lane + 1] <= t));
  Place at{-1, 0, lo >= p.B};
  if (at.behind) return at;
  const int first = p.cu[lo];
  const long long pos = (long long)p.starts[lo] + (t - first);
  if (t >= first && pos >= 0 && pos < (long long)p.max_pages * p.page_size) {
    const unsigned slot = (unsigned)pos / (unsigned)p.page_size;  // pos is below 2^32
    at.page = p.table[lo * p.table_row + slot];
    at.off = (int)((unsigned)pos - slot * (unsigned)p.page_size);
  }
  if (at.page < 0 || at.page >= p.n_pages) at.page = -1;
  return at;
}

// A warp takes a token and `passes` steps of its heads, K's rows and V's: D / 16
// lanes a row, 8 values of each half a lane, since what is done once for a row
// weighs: the issue slots are half full.  16384 tokens of 8 heads of 128, 3 (+ 4 / D) bytes
// a value: written in 19.0 us, read in 20.0, 5.4 and 5.1 TB/s, where adding 1 to
// as many bytes gets 6.2.  (8 values a lane: 22.0 and 20.1; K's and V's rows in
// one list, 20.6 and 20.0: addresses by lane.)  What is missing is the look-up
// before a token's rows can be placed (sequence, start, page: each waits for the
// one before).  Runs of 2 to 4 tokens, looked up at once, are no faster (22.6 and
// 21.0 us): fewer warps then wait for more rows each.
struct Item8 {
  int t, first, end;
};
template <int D>
__device__ __forceinline__ Item8 item_of(const Cache8RowsParams &p) {
  constexpr int kRows = 512 / D;
  const unsigned item = blockIdx.x * 8 + (threadIdx.x >> 5), t = item / (unsigned)p.blocks;
  const int first = (int)(item - t * p.blocks) * p.passes;
  return {(int)t, first, min(first + p.passes, (p.heads + kRows - 1) / kRows)};
}
constexpr int kRowsAhead = 1;  // rows of K and of V that a lane has in flight (2 on 4 CTAs of an SM: write 20.3, read 21.3)

// The lane's place in the rows of K or of V: the packed one, the codes, the scale;
// `step` of each to the rows of the next step.
struct Rows8 {
  __nv_bfloat16 *x;
  uint8_t *codes;
  float *scale;
  long long x_step, codes_step, scale_step;
};
template <int D>
__device__ __forceinline__ Rows8 rows_of8(const Cache8RowsParams &p, bool is_v, int t, int row, int e) {
  Rows8 r;
  constexpr int kRows = 512 / D;
  const long long head = is_v ? p.v_head : p.k_head;
  const CacheStrides &st = is_v ? p.c.vs : p.c.ks, &ss = is_v ? p.c.vss : p.c.kss;
  r.x = (is_v ? p.v + t * p.v_row : p.k + t * p.k_row) + row * head + e;
  r.codes = (is_v ? p.c.v : p.c.k) + row * st.head + e;
  r.scale = (is_v ? p.c.v_scale : p.c.k_scale) + row * ss.head;
  r.x_step = kRows * head;
  r.codes_step = kRows * st.head;
  r.scale_step = kRows * ss.head;
  return r;
}
__device__ __forceinline__ void place_rows(Rows8 &r, const CacheStrides &st, const CacheStrides &ss, Place at) {
  r.codes += at.page * st.page + at.off * st.token;
  r.scale += at.page * ss.page + at.off * ss.token;
}

template <int D>
__device__ __forceinline__ void quantise_row(const uint4 (&x)[2], uint8_t *codes, float *scale, bool first, bool real) {
  constexpr int kLanes = D / 16;
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  // magnitudes in order are bits in order, infinities and NaN above all others
  uint32_t both = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) both = __vmaxu2(both, w[i] & 0x7fff7fffu);
  uint32_t top = max(both & 0xffffu, both >> 16);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool finite = top < 0x7f80u;
  const int f = finite ? scale_field(top) : 1;
  const float inv = pow2_field(254 - f);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = narrow8(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
  uint2 lo = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16), hi = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
  if (!finite) lo = hi = make_uint2(0u, 0u);
  if (!real) return;
  *reinterpret_cast<uint2 *>(codes) = lo;
  *reinterpret_cast<uint2 *>(codes + D / 2) = hi;
  if (first) *scale = finite ? pow2_field(f) : NAN;
}

template <int D>
__global__ void __launch_bounds__(256, 5) dash_cache8_write_kernel(const __grid_constant__ Cache8RowsParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, e = (lane % kLanes) * 8;
  const Item8 it = item_of<D>(p);
  if (it.t >= p.n_tokens) return;
  int row = it.first * kRows + lane / kLanes;
  Rows8 k = rows_of8<D>(p, false, it.t, row, e), v = rows_of8<D>(p, true, it.t, row, e);
  for (int s0 = it.first; s0 < it.end; s0 += kRowsAhead, row += kRowsAhead * kRows) {
    uint4 kx[kRowsAhead][2], vx[kRowsAhead][2];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      kx[u][0] = kx[u][1] = vx[u][0] = vx[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (s0 + u < it.end && row + u * kRows < p.heads) {
        kx[u][0] = *reinterpret_cast<const uint4 *>(k.x);
        kx[u][1] = *reinterpret_cast<const uint4 *>(k.x + D / 2);
        vx[u][0] = *reinterpret_cast<const uint4 *>(v.x);
        vx[u][1] = *reinterpret_cast<const uint4 *>(v.x + D / 2);
      }
      k.x += k.x_step;
      v.x += v.x_step;
    }
    if (s0 == it.first) {  // the rows are on their way meanwhile
      const Place at = place_of(p, it.t, lane);
      if (at.behind) return;
      if (at.page < 0) {
        if (lane == 0) atomicCAS(p.status, 0, kStatusBadPage);
        return;
      }
      place_rows(k, p.c.ks, p.c.kss, at);
      place_rows(v, p.c.vs, p.c.vss, at);
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (s0 + u >= it.end) break;
      const bool real = row + u * kRows < p.heads;
      quantise_row<D>(kx[u], k.codes, k.scale, e == 0, real);
      quantise_row<D>(vx[u], v.codes, v.scale, e == 0, real);
      k.codes += k.codes_step;
      v.codes += v.codes_step;
      k.scale += k.scale_step;
      v.scale += v.scale_step;
    }
  }
}

__device__ __forceinline__ uint4 row_values(uint2 codes, float scale) {
  uint4 w;
  uint32_t *out = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = widen8((i < 2 ? codes.x : codes.y) >> (16 * (i & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&two));
    out[i] = pack_bf16(v.x * scale, v.y * scale);
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(256, 6) dash_cache8_read_kernel(const __grid_constant__ Cache8RowsParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, e = (lane % kLanes) * 8;
  const Item8 it = item_of<D>(p);
  if (it.t >= p.n_tokens) return;
  int row = it.first * kRows + lane / kLanes;
  Rows8 k = rows_of8<D>(p, false, it.t, row, e), v = rows_of8<D>(p, true, it.t, row, e);
  const Place at = place_of(p, it.t, lane);
  const bool none = at.page < 0;  // such rows are zero
  if (none && !at.behind && lane == 0) atomicCAS(p.status, 0, kStatusBadPage);
  place_rows(k, p.c.ks, p.c.kss, at);
  place_rows(v, p.c.vs, p.c.vss, at);
  for (int s0 = it.first; s0 < it.end; s0 += kRowsAhead, row += kRowsAhead * kRows) {
    uint2 kx[kRowsAhead][2], vx[kRowsAhead][2];
    float ks[kRowsAhead], vs[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      kx[u][0] = kx[u][1] = vx[u][0] = vx[u][1] = make_uint2(0u, 0u);
      ks[u] = vs[u] = 0.f;
      if (s0 + u < it.end && row + u * kRows < p.heads && !none) {
        kx[u][0] = *reinterpret_cast<const uint2 *>(k.codes);
        kx[u][1] = *reinterpret_cast<const uint2 *>(k.codes + D / 2);
        vx[u][0] = *reinterpret_cast<const uint2 *>(v.codes);
        vx[u][1] = *reinterpret_cast<const uint2 *>(v.codes + D / 2);
        ks[u] = *k.scale;
        vs[u] = *v.scale;
      }
      k.codes += k.codes_step;
      v.codes += v.codes_step;
      k.scale += k.scale_step;
      v.scale += v.scale_step;
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (s0 + u >= it.end || row + u * kRows >= p.heads) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint4 *>(k.x + i * (D / 2)) = row_values(kx[u][i], ks[u]);
        *reinterpret_cast<uint4 *>(v.x + i * (D / 2)) = row_values(vx[u][i], vs[u]);
      }
      k.x += k.x_step;
      v.x += v.x_step;
    }
  }
}

// A token's rows are one warp's, or, of few tokens, several warps'.
cudaError_t launch_rows(void (*kernel)(const Cache8RowsParams), Cache8RowsParams p, cudaStream_t stream) {
  const int rows = 512 / p.D, steps = (p.heads + rows - 1) / rows, want = 4096;
  p.blocks = p.n_tokens >= want ? 1 : (want + p.n_tokens - 1) / p.n_tokens;
  if (p.blocks > steps) p.blocks = steps;
  p.passes = (steps + p.blocks - 1) / p.blocks;
  p.blocks = (steps + p.passes - 1) / p.passes;
  const long long warps = (long long)p.n_tokens * p.blocks;
  return launch(kernel, (unsigned)((warps + 7) / 8), 256, 0, stream, nullptr, p);
}

// ------------------------------------------------------------------- copy
// As in paged.cu: the pairs travel in the launch's arguments.  Blocks (pair,
// piece) in x, K or V in y; a page's rows are walked 16 bytes a thread, its
// scales one.
template <int N>
struct PairList8 {
  int2 p[N];
};
constexpr int kCopyPairs8 = 3400;  // at most 32764 bytes of arguments

template <int N>
__global__ void __launch_bounds__(256)
    dash_cache8_copy_kernel(const __grid_constant__ PairList8<N> pairs, const Cache8CopyParams p, int pieces) {
  const int vecs = p.D >> 4, rows = p.page_size * p.heads, total = rows * vecs;
  const int pair = blockIdx.x / pieces, piece = blockIdx.x - pair * pieces;
  const int2 pr = pairs.p[pair];
  const bool is_v = blockIdx.y != 0;
  uint8_t *base = is_v ? p.c.v : p.c.k;
  float *scale = is_v ? p.c.v_scale : p.c.k_scale;
  const CacheStrides st = is_v ? p.c.vs : p.c.ks, ss = is_v ? p.c.vss : p.c.kss;
  constexpr int kU = 8;
  for (int x0 = piece * 256 * kU + threadIdx.x; x0 < total; x0 += pieces * 256 * kU) {
    uint4 a[kU];
    long long at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = x0 + 256 * u;
      if (x < total) {
        const int row = x / vecs, tok = row / p.heads;
        at[u] = tok * st.token + (row - tok * p.heads) * st.head + (x - row * vecs) * 16;
        a[u] = *reinterpret_cast<const uint4 *>(base + pr.x * st.page + at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (x0 + 256 * u < total) *reinterpret_cast<uint4 *>(base + pr.y * st.page + at[u]) = a[u];
  }
  for (int x = piece * 256 + threadIdx.x; x < rows; x += pieces * 256) {
    // the shorter of the two inner strides innermost, so that neighbours stay neighbours
    const bool heads_in = ss.head <= ss.token;
    const int in = heads_in ? p.heads : p.page_size, a = x / in, b = x - a * in;
    const long long at = (heads_in ? a : b) * ss.token + (heads_in ? b : a) * ss.head;
    scale[pr.y * ss.page + at] = scale[pr.x * ss.page + at];
  }
}

template <int N>
cudaError_t launch_copy_t(const Cache8CopyParams &p, const int2 *pairs, int n, cudaStream_t stream) {
  PairList8<N> list;
  for (int i = 0; i < n; ++i) list.p[i] = pairs[i];
  const long long total = (long long)p.page_size * p.heads * (p.D / 16);
  const int pieces = (int)((total + 2047) / 2048 < 64 ? (total + 2047) / 2048 : 64);
  return launch(dash_cache8_copy_kernel<N>, dim3(n * pieces, 2), 256, 0, stream, nullptr, list, p, pieces);
}

// ----------------------------------------------------------------- decode
constexpr int kWarps = kDecodeThreads / 32;
constexpr int kTok = 16;              // tokens of a warp's step
constexpr int kStep = kWarps * kTok;  // tokens of the CTA's step
constexpr float kLazy = 256.f;        // growth of a term past its maximum that is left standing

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A step of a warp in its queue: 16 tokens.  Pieces stand lane by lane: of tokens
// g and g + 8 the lane's 16-byte pieces of K, of tokens 2t, 2t + 1, 2t + 8, 2t + 9
// its D / 8 bytes of V (g = lane / 4, t = lane % 4); then 16 scales of K, 16 of V.
template <int D>
struct Queue {
  static constexpr int kStages = 3;
  static constexpr int kK = D / 64, kV = D / 32;  // 16-byte pieces of a K row, words of V
  static constexpr int kVBytes = D / 8;
  static constexpr int oV = 2 * kK * 512, oScale = oV + 4 * 32 * kVBytes;
  static constexpr int kStage = oScale + 128;
  static constexpr int kWarpBytes = kStages * kStage;
};

// Dynamic shared memory: the queues; their place is reused to join the warps, and
// in a cluster for the split's own result.
template <int D, int NT>
struct Dec8 {
  static constexpr int oMl = kWarps * 8 * NT * D * 4, oPart = oMl + kWarps * 8 * NT * 8;
  static constexpr int kJoin = oPart + 16 * (D * 4 + 8);
  static constexpr int kCtas = NT == 1 ? 4 : 2;  // on an SM
  static constexpr int kSmem = kWarps * Queue<D>::kWarpBytes > kJoin ? kWarps * Queue<D>::kWarpBytes : kJoin;
};

// NT tiles of 8 Q heads.
template <int D, int NT, Deal kDeal>
__global__ void __launch_bounds__(kDecodeThreads, Dec8<D, NT>::kCtas)
    dash_decode8_kernel(const __grid_constant__ Decode8Params p) {
  using Q = Queue<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *s_o = reinterpret_cast<float *>(smem);                                       // [warp][head][D]
  float2 *s_ml = reinterpret_cast<float2 *>(smem + Dec8<D, NT>::oMl);                 // [warp][head]
  uint8_t *s_part = smem + Dec8<D, NT>::oPart;
  // the join may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  uint8_t *queue = smem + warp * Q::kWarpBytes;
  Items<kDeal> it;
  for (long long item = blockIdx.x;; item += gridDim.x) {
    const int found = it.find(p, item);
    if (found == 0) break;
    if (found < 0) continue;
    const int b = it.b, split = it.split;
    const int hk = it.rest / p.hblocks, hb = it.rest - hk * p.hblocks;
    const int h0 = hk * p.group + hb * 8 * NT, nh = min(8 * NT, p.group - hb * 8 * NT);
    const int len = decode_len(p, b);
    const int chunk = decode_chunk(len, p.least_chunk), n_splits = max(1, decode_splits(len, p.least_chunk));
    const bool mine = kDeal != kCluster || split < n_splits;  // or the sequence does not have this split of the cluster
    const int begin = split * chunk, end = min(len, begin + chunk);
    const int steps = mine ? (end - begin + kStep - 1) / kStep : 0;
    const int *table = p.table + b * p.table_row;
    const uint8_t *kbase = p.c.k + hk * p.c.ks.head, *vbase = p.c.v + hk * p.c.vs.head;
    const float *ksbase = p.c.k_scale + hk * p.c.kss.head, *vsbase = p.c.v_scale + hk * p.c.vss.head;

    // Where the lane's pieces lie, but for the page and the step's place in it.
    const uint8_t *klane = kbase + g * p.c.ks.token + 16 * t4, *vlane = vbase + 2 * t4 * p.c.vs.token + Q::kVBytes * g;
    const CacheStrides &ss = lane < 16 ? p.c.kss : p.c.vss;
    const float *sbase = lane < 16 ? ksbase : vsbase, *slane = sbase + (lane & 15) * ss.token;
    const int sp = (int)ss.page, st = (int)ss.token;  // only used where they fit

    // Lanes 0-15 know the page of a token of the step, lanes 16-31 likewise.
    auto page_of = [&](int step) -> int {
      const int t = begin + step * kStep + warp * kTok + (lane & 15);
      return t < end ? table[quotient(p.page, t)] : -1;
    };
    // Asks for a step's tokens; returns a bit for each that counts.
    auto load = [&](int step, int slot, int page) -> uint32_t {
      const int t = begin + step * kStep + warp * kTok + (lane & 15);
      const bool inside = step < steps && t < end;
      const bool ok = inside && page >= 0 && page < p.n_pages;
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const uint32_t dst = smem_u32(queue) + slot * Q::kStage;
      if (valid == 0xffffu && p.whole) {
        const int off = t - (lane & 15) - quotient(p.page, t) * p.page_size;
        const uint8_t *kr = wide_add(wide_add(klane, off, (int)p.c.ks.token), page, (int)p.c.ks.page);
        const uint8_t *vr = wide_add(wide_add(vlane, off, (int)p.c.vs.token), page, (int)p.c.vs.page);
        const uint32_t kd = dst + lane * 16, vd = dst + Q::oV + lane * Q::kVBytes;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < Q::kK; ++i)
            cp_async<16>(kd + (r * Q::kK + i) * 512, kr + 8 * r * p.c.ks.token + 64 * i);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          cp_async<Q::kVBytes>(vd + r * 32 * Q::kVBytes, vr + ((r & 1) + 8 * (r >> 1)) * p.c.vs.token);
        cp_async<4>(dst + Q::oScale + lane * 4, wide_add(wide_add(slane, off, st), page, sp));
      } else if (step < steps) {
        if (inside && !ok) atomicCAS(p.status, 0, kStatusBadPage);
        const int off = t - quotient(p.page, t) * p.page_size;
        // a token that does not count is read nowhere: its pieces are zero
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int tok = g + 8 * r, pg = __shfl_sync(0xffffffffu, page, tok), of = __shfl_sync(0xffffffffu, off, tok);
          const bool v = (valid >> tok) & 1u;
          const uint8_t *row = v ? kbase + pg * p.c.ks.page + of * p.c.ks.token + 16 * t4 : p.c.k;
#pragma unroll
          for (int i = 0; i < Q::kK; ++i)
            cp_async_if<16>(dst + (r * Q::kK + i) * 512 + lane * 16, row + (v ? 64 * i : 0), v);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = 2 * t4 + (r & 1) + 8 * (r >> 1);
          const int pg = __shfl_sync(0xffffffffu, page, tok), of = __shfl_sync(0xffffffffu, off, tok);
          const bool v = (valid >> tok) & 1u;
          cp_async_if<Q::kVBytes>(dst + Q::oV + (r * 32 + lane) * Q::kVBytes,
                                  v ? vbase + pg * p.c.vs.page + of * p.c.vs.token + Q::kVBytes * g : p.c.v, v);
        }
        cp_async_if<4>(dst + Q::oScale + lane * 4, ok ? sbase + page * ss.page + off * ss.token : sbase, ok);
      }
      cp_commit();
      return valid;
    };

    constexpr int kAhead = Q::kStages - 1;
    uint64_t fifo = 0;  // 16 bits for each step ahead
    int page = page_of(0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int next = page_of(i + 1);
      fifo |= (uint64_t)load(i, i, page) << (16 * i);
      page = next;
    }

    // Q: head g of each tile, the 16 values of each K piece; its power of two goes into the score's factor
    uint32_t qf[NT][D / 16][2];
    float sc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g;
      const __nv_bfloat16 *q = p.q + b * p.q_batch + (long long)(h0 + row) * p.q_head;
      uint32_t raw[D / 16][2], top = 0;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint2 w = row < nh ? *reinterpret_cast<const uint2 *>(q + 64 * (j >> 2) + 16 * t4 + 4 * (j & 3))
                                 : make_uint2(0u, 0u);
        raw[j][0] = w.x, raw[j][1] = w.y;
#pragma unroll
        for (int i = 0; i < 2; ++i) top = max(top, max(raw[j][i] & 0x7fffu, (raw[j][i] >> 16) & 0x7fffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int f = min(253, 268 - (int)(top >> 7));  // the largest magnitude becomes 2^14 to 2^15
      const float up = top < 0x7f80u ? pow2_field(f) : NAN;  // a head with a NaN or an infinity is all NaN
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[nt][j][i] = pack_f16(__uint_as_float(raw[j][i] << 16) * up, __uint_as_float(raw[j][i] & 0xffff0000u) * up);
      const float down = p.scale_log2 * pow2_field(254 - f);
#pragma unroll
      for (int c = 0; c < 2; ++c) sc[nt][c] = __shfl_sync(0xffffffffu, down, (2 * t4 + c) * 4);
    }

    float acc[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
    // of heads 2 t4 and 2 t4 + 1 of each tile: m, M (-inf: nothing counted yet), 2^(m - M), l of the lane's tokens
    float m[NT][2], M[NT][2], up[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = M[nt][c] = -INFINITY;
        up[nt][c] = NAN;
        l[nt][c] = 0.f;
      }

    int slot = 0;
    for (int step = 0; step < steps; ++step) {
      const int next = page_of(step + kAhead + 1);
      const uint32_t valid = (uint32_t)fifo & 0xffffu;
      fifo = fifo >> 16 | (uint64_t)load(step + kAhead, slot == 0 ? kAhead : slot - 1, page) << (16 * (kAhead - 1));
      page = next;
      cp_wait<kAhead>();
      __syncwarp();  // the scales of other lanes
      const uint8_t *here = queue + slot * Q::kStage;
      slot = slot == kAhead ? 0 : slot + 1;
      const float *scales = reinterpret_cast<const float *>(here + Q::oScale);
      const float ks[2] = {scales[g], scales[g + 8]}, vs[2] = {scales[16 + g], scales[24 + g]};
      float s[NT][4] = {}, s2[NT][4] = {};  // two chains of products
#pragma unroll
      for (int i = 0; i < Q::kK; ++i) {
        const uint4 k0 = *reinterpret_cast<const uint4 *>(here + i * 512 + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4 *>(here + (Q::kK + i) * 512 + lane * 16);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = widen8(w0[w]), a1 = widen8(w1[w]), a2 = widen8(w0[w] >> 16), a3 = widen8(w1[w] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(w & 1 ? s2[nt] : s[nt], a0, a1, a2, a3, qf[nt][4 * i + w][0], qf[nt][4 * i + w][1]);
        }
      }
      // s[nt][2 r + c]: token g + 8 r, head 2 t4 + c
      float pr[NT][4], pv[NT][4], lsum[NT][2], most = 0.f;
      if (valid != 0xffffu) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((valid >> (g + 8 * (e >> 1))) & 1u)) s[nt][e] = s2[nt][e] = -INFINITY;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1, c = e & 1;
          s[nt][e] += s2[nt][e];
          pr[nt][e] = ex2(fmaf(s[nt][e], sc[nt][c] * ks[r], -m[nt][c]));
          pv[nt][e] = pr[nt][e] * (vs[r] * up[nt][c]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          lsum[nt][c] = pr[nt][c] + pr[nt][2 + c];
          most += lsum[nt][c] + (pv[nt][c] + pv[nt][2 + c]);
        }
      }
      // All terms are >= 0: where their sum is within the limit, each is.  A NaN is not within it, and a token that
      // does not count is one here (-inf times its zero scale).
      const bool fast = most <= kLazy;
      if (!__all_sync(0xffffffffu, fast)) {
        // only the heads that need it move, so that a head's bits do not depend on the others
        const float lv[2] = {lg2(vs[0]), lg2(vs[1])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fo[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            bool within = true;
            float x[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int e = 2 * r + c;
              within = within && pr[nt][e] <= kLazy && pv[nt][e] <= kLazy;
              x[r] = (valid >> (g + 8 * r)) & 1u ? s[nt][e] * (sc[nt][c] * ks[r]) : -INFINITY;
            }
            const bool moves = (__ballot_sync(0xffffffffu, !within) & (0x11111111u << t4)) != 0;
            float tm = fmaxf(x[0], x[1]), tM = fmaxf(x[0] + lv[0], x[1] + lv[1]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
              tM = fmaxf(tM, __shfl_xor_sync(0xffffffffu, tM, o));
            }
            fo[c] = 1.f;
            if (!moves) continue;
            const float m1 = fmaxf(m[nt][c], tm), M1 = fmaxf(M[nt][c], tM);
            const float mr = m1 == -INFINITY ? 0.f : m1, Mr = M1 == -INFINITY ? 0.f : M1;
            l[nt][c] *= ex2(m[nt][c] - mr);
            fo[c] = ex2(M[nt][c] - Mr);
            m[nt][c] = m1;
            M[nt][c] = M1;
            // a factor that 32 bits cannot hold stays NaN, and every step comes here
            up[nt][c] = fabsf(m1 - M1) < 100.f ? ex2(m1 - M1) : NAN;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              pr[nt][2 * r + c] = ex2(x[r] - mr);
              pv[nt][2 * r + c] = ex2(x[r] + lv[r] - Mr);
            }
            lsum[nt][c] = pr[nt][c] + pr[nt][2 + c];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][i][e] *= fo[e & 1];
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) l[nt][c] += lsum[nt][c];
        pb[nt][0] = transpose8x8(pack_f16(pv[nt][0], pv[nt][1]));
        pb[nt][1] = transpose8x8(pack_f16(pv[nt][2], pv[nt][3]));
      }
      uint32_t v[4][Q::kV];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t *at = here + Q::oV + (r * 32 + lane) * Q::kVBytes;
        if (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4 *>(at);
          v[r][0] = w.x, v[r][1] = w.y, v[r][Q::kV - 2] = w.z, v[r][Q::kV - 1] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(at);
          v[r][0] = w.x, v[r][1] = w.y;
        }
      }
#pragma unroll
      for (int w = 0; w < Q::kV; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // dims 2 half, 2 half + 1 of the word: {first, second token} pairs of codes
          const uint32_t y0 = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
          const uint32_t y1 = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
          const uint32_t a0 = widen8(y0), a1 = widen8(y0 >> 16), a2 = widen8(y1), a3 = widen8(y1 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][2 * w + half], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      __syncwarp();  // every lane has read the slot that the next step fills
    }
    cp_wait<0>();
    __syncthreads();  // every warp has left its queue

    // ---- each warp's average with its maximum and sum, then their join
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
        const int row = 8 * nt + 2 * t4 + c;
        const float f = l[nt][c] == 0.f ? 0.f : ex2(M[nt][c] - m[nt][c]), inv = inverse_sum(l[nt][c]);
        float *o = s_o + (warp * 8 * NT + row) * D + (D / 8) * g;
#pragma unroll
        for (int w = 0; w < Q::kV; ++w)
          *reinterpret_cast<float4 *>(o + 4 * w) =
              make_float4(acc[nt][2 * w][c] * inv * f, acc[nt][2 * w][2 + c] * inv * f,
                          acc[nt][2 * w + 1][c] * inv * f, acc[nt][2 * w + 1][2 + c] * inv * f);
        if (g == 0) s_ml[warp * 8 * NT + row] = make_float2(m[nt][c], l[nt][c]);
      }
    __syncthreads();
    constexpr int kVec = D / 4;
    using J = Join<D>;
    for (int y = threadIdx.x; mine && y < nh * kVec; y += kDecodeThreads) {
      const int row = y / kVec, c = (y - row * kVec) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w * 8 * NT + row].x);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float fw = J::weight(s_ml[w * 8 * NT + row], ref);
        ll += fw;
        J::add(o, fw, *reinterpret_cast<const float4 *>(s_o + (w * 8 * NT + row) * D + c));
      }
      const int h = h0 + row;
      if (n_splits == 1) {
        J::write(p, b, h, c, o, mm, ll);
      } else {
        const float inv = inverse_sum(ll);
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (kDeal == kCluster) {
          float *part = reinterpret_cast<float *>(s_part);  // [16][D], then [16] {maximum, sum}
          *reinterpret_cast<float4 *>(part + row * D + c) = o;
          if (c == 0) reinterpret_cast<float2 *>(part + 16 * D)[row] = make_float2(mm, ll);
        } else {
          const size_t at = ((size_t)b * p.Hq + h) * p.max_splits + split;
          *reinterpret_cast<float4 *>(p.part_o + at * D + c) = o;
          if (c == 0) p.part_ml[at] = make_float2(mm, ll);
        }
      }
    }
    if (kDeal == kCluster) {
      if (n_splits > 1) join_cluster<D>(p, s_part, b, h0, nh, split, n_splits);  // the same in every CTA of the cluster
      break;
    }
    __syncthreads();  // shared memory is free for the next item
  }
}

template <int D, int NT>
cudaError_t launch_decode_t(const Decode8Params &p, int num_sms, cudaStream_t stream) {
  constexpr int kSmem = Dec8<D, NT>::kSmem;
  const long long items = (long long)p.B * p.max_splits * p.Hkv * p.hblocks;
  if (decode_clustered(p.B, p.Hq, p.max_splits)) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.max_splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    return launch(dash_decode8_kernel<D, NT, kCluster>, (int)items, kDecodeThreads, kSmem, stream, &attr, p);
  }
  const int resident = Dec8<D, NT>::kCtas * num_sms;
  const bool all = items <= resident;
  if constexpr (NT == 1) {
    // An item of the other form costs as much as two or three of its tiles, however short, so sequences that cannot be
    // long stay here: at D = 64 up to 512 tokens (256 of 256, 32 heads on 8: 27.9 us against 35.0; 64 of 768 on 16 K/V
    // heads 38.6 and 36.1), at D = 128 up to 64 (500 of 64: 43.0 and 49.3; 256 of 128: 30.8 and 27.6).
    if (!all && p.max_pages * p.page_size > (D == 64 ? 512 : 64)) {
      Decode8Params q = p;
      q.least_chunk = 1024;  // an item's start and end cost as much as two tiles of 128 tokens
      const cudaError_t e = launch_decode8_wide(D, q, num_sms, stream);
      return e != cudaSuccess || q.max_splits <= 1 ? e : launch_decode_join(D, q, stream);
    }
  }
  const cudaError_t e = launch(all ? dash_decode8_kernel<D, NT, kPlain> : dash_decode8_kernel<D, NT, kScan>, all ? (int)items : resident, kDecodeThreads, kSmem, stream, nullptr, p);
  return e != cudaSuccess || p.max_splits <= 1 ? e : launch_decode_join(D, p, stream);
}

template <int D, int NT>
cudaError_t prepare_t() {
  auto set = [](void (*kernel)(const Decode8Params)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Dec8<D, NT>::kSmem);
  };
  cudaError_t e = set(dash_decode8_kernel<D, NT, kPlain>);
  if (e == cudaSuccess) e = set(dash_decode8_kernel<D, NT, kScan>);
  if (e == cudaSuccess) e = set(dash_decode8_kernel<D, NT, kCluster>);
  return e;
}

}  // namespace

cudaError_t prepare_cache8() {
  cudaFuncAttributes fa;
  for (auto kernel : {dash_cache8_write_kernel<64>, dash_cache8_write_kernel<128>, dash_cache8_read_kernel<64>,
                      dash_cache8_read_kernel<128>})
    if (const cudaError_t e = cudaFuncGetAttributes(&fa, kernel)) return e;
  cudaError_t e = prepare_decode8_wide();
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, dash_cache8_copy_kernel<64>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, dash_cache8_copy_kernel<kCopyPairs8>);
  if (e == cudaSuccess) e = prepare_t<64, 1>();
  if (e == cudaSuccess) e = prepare_t<64, 2>();
  if (e == cudaSuccess) e = prepare_t<128, 1>();
  return e != cudaSuccess ? e : prepare_t<128, 2>();
}

cudaError_t launch_decode8(int D, const Decode8Params &p, int num_sms, cudaStream_t stream) {
  const bool small = p.group <= 8;
  if (D == 64) return small ? launch_decode_t<64, 1>(p, num_sms, stream) : launch_decode_t<64, 2>(p, num_sms, stream);
  return small ? launch_decode_t<128, 1>(p, num_sms, stream) : launch_decode_t<128, 2>(p, num_sms, stream);
}

cudaError_t launch_cache8_write(const Cache8RowsParams &p, cudaStream_t stream) {
  return launch_rows(p.D == 64 ? dash_cache8_write_kernel<64> : dash_cache8_write_kernel<128>, p, stream);
}

cudaError_t launch_cache8_read(const Cache8RowsParams &p, cudaStream_t stream) {
  return launch_rows(p.D == 64 ? dash_cache8_read_kernel<64> : dash_cache8_read_kernel<128>, p, stream);
}

cudaError_t launch_cache8_copy(const Cache8CopyParams &p, const int2 *pairs, int n, cudaStream_t stream) {
  for (int i = 0; i < n; i += kCopyPairs8) {
    const int k = n - i < kCopyPairs8 ? n - i : kCopyPairs8;
    const cudaError_t e =
        k <= 64 ? launch_copy_t<64>(p, pairs + i, k, stream) : launch_copy_t<kCopyPairs8>(p, pairs + i, k, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dash
