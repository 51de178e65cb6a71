// Packed, grouped-head attention backward for sm_103a, deterministic by
// construction: every gradient element is summed in one order, by one CTA, or,
// where a KV tile's Q tiles are dealt to several, by each over its part and then
// over the parts in turn.
//
//   P = 2^(scale log2(e) q.k - LSE log2(e)),  delta_i = dO_i . O_i,
//   dS = P (dO V^T - delta),
//   dQ = scale dS K,   dK = scale sum_heads dS^T Q,   dV = sum_heads P^T dO.
//
// Two kernels (and a third that adds up parts), each with its own P and dS: dQ
// walks the KV tiles of a Q tile, dK/dV the Q tiles (of every Q head of the
// group) of a KV tile.  That makes seven products of 128 x 128 x D a tile pair where one kernel for all three
// gradients makes five, but nothing crosses a CTA: no 32-bit dQ accumulator in
// memory, no order to enforce between CTAs, no wait of one CTA for another, and
// dQ's place in tensor memory lets the products run under the softmax.  The
// one-kernel form (tiles of dQ reduced in the order of a schedule) ran a
// training batch of 16384 tokens (16 heads on 4, D = 128) in 737 us and long
// documents at D = 64 (32 heads on 8) in 2151 us; this one takes 416 (dQ 176,
// dK and dV 240) and 1216 (480 and 715), each replayed from a graph, and 444 and
// 1238 through the call with fresh inputs.  The MMAs keep the tensor pipe 70 %
// busy at D = 128; what is left is the chain from one tile's scores to the next
// tile's (waits, exponentials) and, for dQ, shared memory's bandwidth, and at
// D = 64 the softmax warps' instructions and waits: with next to no MMAs dK/dV
// would still take 79 % of its time, without its exponentials as long as now.
//
// Warps of both kernels: sixteen turn scores into P and dS (a thread owns 32
// columns of a row of the accumulator), then X, Y and Z, which issue the MMAs, one that loads, and four that write the
// last item's results, clear rows past a sequence's end that a product sums over
// and, for dQ, make the next item's delta.  Several warps issue, because a wait
// answers about 100 clocks after the MMAs in front of it, which another warp's
// MMAs cover.
//
// P and dS are rounded to bf16 as MMA operands, once each; everything else is
// held in 32 bits until the gradients' own rounding.
#include <cuda_runtime.h>

#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kSoft = 16;                // softmax warps
constexpr int kThreads = (kSoft + 8) * 32;
constexpr int kCols = 128 / (kSoft / 4);  // columns of a softmax thread
constexpr int kRegsLaunch = 80, kRegsSoft = 88, kRegsOther = 64, kRegsOut = 64;
static_assert(kCols == 32 && kRegsSoft * kSoft / 4 + kRegsOther + kRegsOut <= kRegsLaunch * (kSoft + 8) / 4,
              "register split exceeds the CTA's allocation");

__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t dup2(float a) { return pack2(__float_as_uint(a), __float_as_uint(a)); }

template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1;
    }
  }
};

template <class T>
__device__ __forceinline__ T load_item(const T *p) {
  T it;
  int4 *d = reinterpret_cast<int4 *>(&it);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 16; ++i) d[i] = __ldg(reinterpret_cast<const int4 *>(p) + i);
  return it;
}

// Clears the rows first .. 127 of a swizzled tile (a row is 128 bytes of each
// 64-column panel, whatever the swizzle does inside it).
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int first, int lane) {
  for (int x = first * 8 + lane; x < kPackedTile * 8; x += 32)
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn)
      *reinterpret_cast<uint4 *>(tile + pn * (128 * 128) + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 accumulator columns of a row, scaled and rounded, in registers: tensor
// memory is free before the last of them go to global memory.
struct OutRow {
  uint32_t w[16];
  __device__ __forceinline__ void read(uint32_t taddr, float scale) {
    uint32_t r[32];
    tmem_ld32(taddr, r);
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      w[e >> 1] = pack_bf16(scale * __uint_as_float(r[e]), scale * __uint_as_float(r[e + 1]));
  }
  __device__ __forceinline__ void write(__nv_bfloat16 *out, bool wide) const {
    st_32b(out, w, wide);
    st_32b(out + 16, w + 8, wide);
  }
};

// A whole row in 32 bits, as one part of a sum.
template <int D>
__device__ __forceinline__ void write_part(uint32_t taddr, float *out, bool wide) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c, r);
#pragma unroll
    for (int e = 0; e < 32; e += 8) st_32b(out + c + e, r + e, wide);
  }
}

// P and dS replace the scores they come from: the kCols columns of a thread
// pack into the first half of their own place, which the same thread has read,
// so threads of one row never race.  K step kk (16 columns) of the MMA that
// reads them:
__device__ __forceinline__ constexpr uint32_t packed_col(int kk) {
  return 16 * kk / kCols * kCols + 16 * kk % kCols / 2;
}

// Shared parts of the two kernels.
template <int D>
struct Tile {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kBytes = 128 * D * 2;
  static constexpr uint32_t kPanel = 128 * 128;
  // k-step offset of a K-major operand, in descriptor units
  static __device__ __forceinline__ constexpr uint32_t kmajor(int kk) {
    return ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
  }
  static __device__ __forceinline__ void load(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int row, int head) {
    for (int pn = 0; pn < kPanels; ++pn) tma_load_3d(dst + pn * kPanel, m, bar, pn * 64, row, head);
  }
};

// ------------------------------------------------------------------- dQ
// Per KV tile j:   X: dP(j+1) = dO V^T     Y: dQ += dS(j) K     Z: S(j+2) = Q K^T
// once the softmax warps have dP(j) in registers (X), dS(j) is in tensor memory
// (Y) and dQ(j) has read dS(j), whose place S(j+2) takes (Z).
// Tensor memory: S and dS in two buffers at 0 and 128, dP at 256, dQ at 384.  V
// rows past the sequence's end reach dP only, whose columns there are replaced;
// K rows there are summed over and are cleared.
template <int D>
struct DqCfg : Tile<D> {
  static constexpr int kQ = D == 128 ? 1 : 2, kK = D == 128 ? 3 : 5, kV = D == 128 ? 2 : 4;  // stages
  static constexpr uint32_t oQ = 0, oDO = kQ * Tile<D>::kBytes, oK = 2 * kQ * Tile<D>::kBytes;
  static constexpr uint32_t oV = oK + kK * Tile<D>::kBytes;
  static constexpr uint32_t oSTAT = oV + kV * Tile<D>::kBytes;  // [2][128] {-lse2, -delta}
  static constexpr uint32_t oBAR = oSTAT + 2 * 128 * 8;
  enum {
    // S and dS have a barrier per buffer: a warp may be a tile ahead of another.  So have the tails: S, which
    // asks for them, is up to two tiles (and items) ahead of dQ, which waits for them.
    bSFull, bSEmpty = bSFull + 2, bDpFull = bSEmpty + 2, bRead, bDsFull, bOFull = bDsFull + 2, bOEmpty, bTail,
    bFixed = bTail + 2, bFinalX = bFixed + 2, bFinalY, bFinalZ, bStat,
    bKFull = bStat + 2, bKEmpty = bKFull + kK, bVFull = bKEmpty + kK, bVEmpty = bVFull + kV,
    bQFull = bVEmpty + kV, bQEmpty = bQFull + kQ, bDOFull = bQEmpty + kQ, bDOEmpty = bDOFull + kQ,
    kBars = bDOEmpty + kQ
  };
  static constexpr uint32_t oMISC = oBAR + kBars * 8;
  static constexpr uint32_t kSmem = oMISC + 16;
  static constexpr uint32_t cDP = 256, cDQ = 384;
};
static_assert(DqCfg<128>::kSmem <= 232448 && DqCfg<64>::kSmem <= 232448, "shared memory of one CTA");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dash_packed_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                          const PackedBwdParams p) {
  using C = DqCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = warp_id(), lane = threadIdx.x & 31;
  const int role = warp - kSoft;  // below 0: softmax; 0 X, 1 Y, 2 loads, 3 Z, 4-7 delta and the results
  // dK/dV's CTAs may take the SMs that this kernel leaves; they wait for its end before they read the stats
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::oBAR);
  float2 *stat = reinterpret_cast<float2 *>(smem + C::oSTAT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::oMISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::oMISC + 4);
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemMisaligned);
    return;
  }
  if (threadIdx.x == 0) {
    for (int b = 0; b < C::kBars; ++b)
      mbar_init(&bars[b], b >= C::bRead && b < C::bDsFull + 2                     ? kSoft
                          : b == C::bOEmpty || b == C::bStat || b == C::bStat + 1 ? 4
                                                                                  : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (role == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, p.status, (uint64_t)p.spin_limit_ns};
  const int i_begin = p.dq_off[blockIdx.x], i_end = p.dq_off[blockIdx.x + 1];

  if (role >= 4) {
    // ------------------------------------------------- delta and epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    const int sub = warp & 3;
    // A warp makes the stats of its 32 rows: D / 16 lanes of 32 bytes a row, in
    // rounds of loads that the registers hold.  The rows come from memory (nobody
    // else has read O), so the item behind asks L2 for them (128 documents of 128
    // tokens at D = 128: 75 us in all, 81 without that).
    auto ask = [&](int i) {
      const PackedDqItem it = load_item(p.dq_items + i);
      const int r = sub * 32 + lane;
      if (r < it.rows) {
        const __nv_bfloat16 *o = p.o + (it.row0 + r) * p.o_row + it.head * p.o_head;
        const __nv_bfloat16 *d = p.dout + (it.row0 + r) * p.do_row + it.head * p.do_head;
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(o + c));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(d + c));
        }
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.lse + it.head * p.lse_head + it.row0 + r));
      }
    };
    auto make_stats = [&](int i) {
      const PackedDqItem it = load_item(p.dq_items + i);
      constexpr int kLanes = D / 16, kRows = 32 / kLanes, kU = 2, kRound = kRows * kU;
      const int li = lane % kLanes, rs = lane / kLanes;
      const int mine = sub * 32 + lane, first = sub * 32 + rs;
      const __nv_bfloat16 *o = p.o + (it.row0 + first) * p.o_row + it.head * p.o_head + li * 16;
      const __nv_bfloat16 *d = p.dout + (it.row0 + first) * p.do_row + it.head * p.do_head + li * 16;
      float nl = __int_as_float(0xff800000), nd = 0.f;  // of this lane's row
      if (mine < it.rows) nl = -p.lse[it.head * p.lse_head + it.row0 + mine] * 1.4426950408889634f;
#pragma unroll 1
      for (int row = 0; row < 32; row += kRound, o += kRound * p.o_row, d += kRound * p.do_row) {
        uint32_t a[kU][8], b[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (first + row + u * kRows < it.rows) {
            ld_32b(o + u * kRows * p.o_row, a[u], p.wide_in);
            ld_32b(d + u * kRows * p.do_row, b[u], p.wide_in);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) a[u][x] = b[u][x] = 0u;
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const __nv_bfloat162 *pa = reinterpret_cast<const __nv_bfloat162 *>(a[u]);
          const __nv_bfloat162 *pb = reinterpret_cast<const __nv_bfloat162 *>(b[u]);
          float sum = 0.f;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float2 fa = __bfloat1622float2(pa[x]), fb = __bfloat1622float2(pb[x]);
            sum = fmaf(fa.x, fb.x, sum);
            sum = fmaf(fa.y, fb.y, sum);
          }
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          // every lane of a row has its sum: hand it to the lane that keeps the row
          const int at = lane - row - u * kRows;
          const float got = __shfl_sync(0xffffffffu, sum, (at & (kRows - 1)) * kLanes);
          if (at >= 0 && at < kRows) nd = -got;
        }
      }
      stat[(i & 1) * 128 + mine] = make_float2(nl, nd);
      float *out = p.stats + ((size_t)it.head * p.n_tiles + it.tile) * 256;
      out[mine] = nl;
      out[128 + mine] = nd;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[C::bStat + (i & 1)]);
    };
    const int L = sub * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(sub * 32) << 16) + C::cDQ;
    uint32_t ph = 0, loads = 0, tail_ph = 0, tail = 0;
    if (i_begin < i_end) make_stats(i_begin);
    if (i_begin + 1 < i_end) ask(i_begin + 1);
    for (int i = i_begin; i < i_end; ++i) {
      // stats (i + 1) & 1 were read when item i - 1 began, which is over
      if (i + 1 < i_end) make_stats(i + 1);
      if (i + 2 < i_end) ask(i + 2);
      const PackedDqItem it = load_item(p.dq_items + i);
      loads += it.nkv;
      if (it.nkv * kPackedTile > it.kv_len) {  // K rows past the end in the item's last tile
        if (sub == 0) {
          mbar_wait(&bars[C::bTail + tail], tail_ph, g);
          if (!warp_aborted(g))
            clear_rows<D>(smem + C::oK + (loads - 1) % C::kK * C::kBytes, it.kv_len - (it.nkv - 1) * kPackedTile, lane);
          if (lane == 0) mbar_arrive(&bars[C::bFixed + tail]);
        }
        tail_ph ^= tail;
        tail ^= 1;
      }
      bool ok = mbar_wait(&bars[C::bOFull], ph, g);
      ph ^= 1;
      __syncwarp();
      tc_fence_after();
      ok &= L < it.rows;
      __nv_bfloat16 *to = p.dq + ((long long)it.row0 + L) * p.dq_row + it.head * p.dq_head;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        OutRow out;
        out.read(tq + c, p.scale);
        if (c + 32 == D) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[C::bOEmpty]);
        }
        if (ok) out.write(to + c, p.wide_dq);
        __syncwarp();
      }
    }
  } else if (role >= 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    uint32_t lead = elect_one();
    auto wait = [&](int bar, uint32_t ph) {
      if (!mbar_wait(&bars[bar], ph, g)) lead = 0;
    };
    if (role == 2 && lane == 0) {
      // -------------------------------------------------------------- TMA
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmDO);
      Ring<C::kK> rk;
      Ring<C::kV> rv;
      Ring<C::kQ> rq;
      uint32_t nq = 0, nk = 0, nv = 0;
      bool live = true;
      auto load = [&](int full, int empty, uint32_t ph, uint32_t at, const CUtensorMap *m, int row, int head) {
        live = live && mbar_wait(&bars[empty], ph ^ 1, g);
        if (!live) return 0u;
        mbar_arrive_expect_tx(&bars[full], C::kBytes);
        C::load(smem + at, m, &bars[full], row, head);
        return 1u;
      };
      uint32_t ndo = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const PackedDqItem it = load_item(p.dq_items + i);
        const int kvh = it.head / p.group;
        nq += load(C::bQFull + rq.st, C::bQEmpty + rq.st, rq.ph, C::oQ + rq.st * C::kBytes, &tmQ, it.row0, it.head);
        for (int j = 0; j < it.nkv; ++j) {
          const int row = it.kv_row0 + j * kPackedTile;
          nk += load(C::bKFull + rk.st, C::bKEmpty + rk.st, rk.ph, C::oK + rk.st * C::kBytes, &tmK, row, kvh);
          rk.next();
          if (j == 0)  // the last dP before needs dO longer than the last S needs Q
            ndo += load(C::bDOFull + rq.st, C::bDOEmpty + rq.st, rq.ph, C::oDO + rq.st * C::kBytes, &tmDO, it.row0,
                        it.head);
          nv += load(C::bVFull + rv.st, C::bVEmpty + rv.st, rv.ph, C::oV + rv.st * C::kBytes, &tmV, row, kvh);
          rv.next();
        }
        rq.next();
      }
      // copies still in flight land before the CTA exits
      auto drain = [&](int bar, uint32_t n, uint32_t stages) {
        for (uint32_t s = 0; s < stages; ++s) {
          const uint32_t f = n / stages + (s < n % stages ? 1u : 0u);
          if (f) mbar_drain(&bars[bar + s], (f - 1) & 1, g.limit_ns);
        }
      };
      drain(C::bQFull, nq, C::kQ);
      drain(C::bDOFull, ndo, C::kQ);
      drain(C::bKFull, nk, C::kK);
      drain(C::bVFull, nv, C::kV);
    } else if (role == 0) {
      // ------------------------------------------------------- X: dP
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      const uint64_t ddo0 = sw128_desc(smem_u32(smem + C::oDO), 16, 1024);
      const uint64_t dv0 = sw128_desc(smem_u32(smem + C::oV), 16, 1024);
      Ring<C::kV> rv;
      Ring<C::kQ> rq;
      uint32_t read_ph = 1;
      for (int i = i_begin; i < i_end; ++i) {
        const int nkv = p.dq_items[i].nkv;
        wait(C::bDOFull + rq.st, rq.ph);
        const uint64_t ddo = ddo0 + ((rq.st * C::kBytes) >> 4);
        for (int j = 0; j < nkv; ++j) {
          wait(C::bVFull + rv.st, rv.ph);
          wait(C::bRead, read_ph);  // the dP before is in registers
          read_ph ^= 1;
          tc_fence_after();
          const uint64_t dv = dv0 + ((rv.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_if(lead, tmem + C::cDP, ddo + C::kmajor(kk), dv + C::kmajor(kk), idS, kk > 0);
          tc_commit_if(lead, &bars[C::bDpFull]);
          tc_commit_if(lead, &bars[C::bVEmpty + rv.st]);
          rv.next();
        }
        tc_commit_if(lead, &bars[C::bDOEmpty + rq.st]);
        rq.next();
      }
      // every MMA has completed before tensor memory is released (at once if none was issued)
      tc_commit_if(elect_one(), &bars[C::bFinalX]);
      mbar_drain(&bars[C::bFinalX], 0, g.limit_ns);
    } else if (role == 1) {
      // ------------------------------------------------------- Y: dQ
      constexpr uint32_t idQ = idesc_bf16(128, D, 0, 1);
      const uint64_t dk0 = sw128_desc(smem_u32(smem + C::oK), C::kPanel, 1024);
      Ring<C::kK> rk;
      uint32_t ds_ph = 0, o_ph = 1, fix_ph = 0, fix = 0, buf = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const int nkv = p.dq_items[i].nkv;
        const bool ragged = nkv * kPackedTile > p.dq_items[i].kv_len;
        for (int j = 0; j < nkv; ++j) {
          wait(C::bKFull + rk.st, rk.ph);
          if (ragged && j + 1 == nkv) {
            wait(C::bFixed + fix, fix_ph);
            fix_ph ^= fix;
            fix ^= 1;
          }
          if (j == 0) {  // the item before has been written out
            wait(C::bOEmpty, o_ph);
            o_ph ^= 1;
          }
          wait(C::bDsFull + buf, ds_ph);
          ds_ph ^= buf;  // both buffers' parity, which changes after the second
          tc_fence_after();
          const uint64_t dk = dk0 + ((rk.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_if(lead, tmem + C::cDQ, tmem + buf * 128 + packed_col(kk), dk + ((kk * 2048) >> 4), idQ,
                      (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit_if(lead, &bars[C::bSEmpty + buf]);
          tc_commit_if(lead, &bars[C::bKEmpty + rk.st]);
          if (j + 1 == nkv) tc_commit_if(lead, &bars[C::bOFull]);
          buf ^= 1;
          rk.next();
        }
      }
      tc_commit_if(elect_one(), &bars[C::bFinalY]);
      mbar_drain(&bars[C::bFinalY], 0, g.limit_ns);
    } else if (role == 3) {
      // ------------------------------------- Z: S, from one item into the next
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      const uint64_t dq0 = sw128_desc(smem_u32(smem + C::oQ), 16, 1024);
      const uint64_t dk0 = sw128_desc(smem_u32(smem + C::oK), 16, 1024);
      Ring<C::kK> rk;
      Ring<C::kQ> rq;
      uint32_t e_ph = 1, tail = 0, buf = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const int nkv = p.dq_items[i].nkv;
        const bool ragged = nkv * kPackedTile > p.dq_items[i].kv_len;
        wait(C::bQFull + rq.st, rq.ph);
        const uint64_t dq = dq0 + ((rq.st * C::kBytes) >> 4);
        for (int j = 0; j < nkv; ++j) {
          wait(C::bKFull + rk.st, rk.ph);
          wait(C::bSEmpty + buf, e_ph);
          e_ph ^= buf;
          // it has landed: the rows past the end may be cleared, while S reads them (their columns are replaced).
          // Not before the wait, by which the tail before the last has been dealt with: two barriers hold two.
          if (ragged && j + 1 == nkv) {
            if (lead) mbar_arrive(&bars[C::bTail + tail]);
            tail ^= 1;
          }
          tc_fence_after();
          const uint64_t dk = dk0 + ((rk.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_if(lead, tmem + buf * 128, dq + C::kmajor(kk), dk + C::kmajor(kk), idS, kk > 0);
          tc_commit_if(lead, &bars[C::bSFull + buf]);
          buf ^= 1;
          rk.next();
        }
        tc_commit_if(lead, &bars[C::bQEmpty + rq.st]);
        rq.next();
      }
      tc_commit_if(elect_one(), &bars[C::bFinalZ]);
      mbar_drain(&bars[C::bFinalZ], 0, g.limit_ns);
    }
  } else {
    // ------------------------------------------------------------- dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int sub = warp & 3, c0 = (warp >> 2) * kCols;  // its columns of S and dP
    const int L = sub * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16) + c0;
    const uint64_t sc2 = dup2(p.scale_log2);
    uint32_t n = 0;       // tiles before this one; its parities give the buffers and the phases
    uint32_t st_ph = 0;   // a bit per stats buffer
    for (int i = i_begin; i < i_end; ++i) {
      const PackedDqItem it = load_item(p.dq_items + i);
      mbar_wait(&bars[C::bStat + (i & 1)], (st_ph >> (i & 1)) & 1, g);
      st_ph ^= 1u << (i & 1);
      const float2 ls = stat[(i & 1) * 128 + L];
      const uint64_t nl2 = dup2(ls.x), nd2 = dup2(ls.y);
      // the columns of this thread that are valid, counted on through the tiles
      int cols = (p.causal ? min(it.kv_len, it.q0 + L + 1) : it.kv_len) - c0;
      for (int left = it.nkv; left > 0; --left, ++n, cols -= kPackedTile) {
        const uint32_t buf = n & 1;
        mbar_wait(&bars[C::bSFull + buf], n >> 1 & 1, g);
        mbar_wait(&bars[C::bDpFull], n & 1, g);
        __syncwarp();
        tc_fence_after();
        uint32_t x[32], y[32];
        tmem_ld32_nowait(tl + buf * 128, x);
        tmem_ld32_nowait(tl + C::cDP, y);
        tmem_wait_ld();
        reg_order32(x);
        reg_order32(y);
        tc_fence_before();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a, b;
          unpack2(fma2(pack2(x[e], x[e + 1]), sc2, nl2), a, b);
          x[e] = __float_as_uint(ex2(a));
          x[e + 1] = __float_as_uint(ex2(b));
        }
        auto make_ds = [&](int from) {
#pragma unroll
          for (int e = from; e < from + 16; e += 2) {
            float a, b;
            unpack2(mul2(pack2(x[e], x[e + 1]), add2(pack2(y[e], y[e + 1]), nd2)), a, b);
            y[e] = __float_as_uint(a);
            y[e + 1] = __float_as_uint(b);
          }
        };
        make_ds(0);
        // S and dP have been in registers for long, but X is told now: the next dP
        // then starts shortly before dQ, not in the middle of the exponentials
        // (16384 tokens, 16 heads on 4: 861 us against 930 at D = 128, 594
        // against 642 at D = 64; behind the rounding it is too late, 1058 and
        // 750).  The registers pass through the statements in this order.
        reg_order32(x);
        reg_order32(y);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::bRead]);
        make_ds(16);
        if (__any_sync(0xffffffffu, cols < kCols)) {
          // selected, not multiplied: dP there may come from rows of another sequence
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= cols) y[e] = 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) pk[e >> 1] = pack_bf16(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
        tmem_st16(tl + buf * 128, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::bDsFull + buf]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (role == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- dK and dV
// The accumulators' lanes are KV rows.  Per Q tile i (of every head):
//   X: dV += P^T(i) dO, S^T(i+1) = K Q^T     Y: dK += dS^T(i) Q, dP^T(i+1) = V dO^T
// (with two S buffers a third warp, Z, issues S^T(i+2) once dV(i) has read P).
// P^T and dS^T replace S^T and dP^T in tensor memory (S at 0, dP at 128, dV at
// 256, dK at 256 + D; at D = 64 two S at 0 and 128 and the others behind).
// Rows of dO (for dV) and of Q (for dK) past the sequence's end are summed over
// and cleared first; K and V rows there only reach accumulator rows that are
// not written.
template <int D>
struct DkvCfg : Tile<D> {
  static constexpr int kQ = D == 128 ? 3 : 4, kDO = D == 128 ? 2 : 4, kSt = D == 128 ? 2 : 4;  // stages
  // Buffers of S^T: a second one, where tensor memory has room, lets the next
  // score run before dV has read this P.
  static constexpr int kS = D == 128 ? 1 : 2;
  // With one buffer, S -> P -> dV -> S is the chain that sets the pace, and X
  // and Y take turns so that each pair of products runs in one piece.  Passing
  // the turn is an arrival on the barrier that counts P (for X) or dS (for Y):
  // one wait answers for both.
  static constexpr bool kTurns = kS == 1;
  static constexpr uint32_t oK = 0, oV = Tile<D>::kBytes, oQ = 2 * Tile<D>::kBytes;
  static constexpr uint32_t oDO = oQ + kQ * Tile<D>::kBytes;
  static constexpr uint32_t oSTAT = oDO + kDO * Tile<D>::kBytes;  // [kSt][2][128]
  static constexpr uint32_t oBAR = oSTAT + kSt * 1024;
  enum {
    bKFull, bKEmpty, bVFull, bVEmpty, bSFull, bSEmpty = bSFull + kS, bPFull = bSEmpty + kS, bDpFull = bPFull + kS,
    bDsFull, bDvFull, bDkFull, bDvEmpty, bDkEmpty, bTailQ, bFixedQ, bTailDO, bFixedDO, bFinalX, bFinalY, bFinalZ,
    bQFull, bQEmpty = bQFull + kQ, bDOFull = bQEmpty + kQ, bDOEmpty = bDOFull + kDO, bStFull = bDOEmpty + kDO,
    bStEmpty = bStFull + kSt, kBars = bStEmpty + kSt
  };
  static constexpr uint32_t oMISC = oBAR + kBars * 8;
  static constexpr uint32_t kSmem = oMISC + 16;
  static constexpr uint32_t cDP = 128 * kS, cDV = cDP + 128, cDK = cDV + D;
  static_assert(cDK + D <= 512, "tensor memory");
};
static_assert(DkvCfg<128>::kSmem <= 232448 && DkvCfg<64>::kSmem <= 232448, "shared memory of one CTA");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dash_packed_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                           const PackedBwdParams p) {
  using C = DkvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = warp_id(), lane = threadIdx.x & 31;
  const int role = warp - kSoft;  // below 0: softmax; 0 X, 1 Y, 2 loads, 3 Z, 4-7 write the results
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::oBAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::oMISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::oMISC + 4);
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemMisaligned);
    return;
  }
  if (threadIdx.x == 0) {
    for (int b = 0; b < C::kBars; ++b) {
      const bool turn = (b >= C::bPFull && b < C::bDpFull) || b == C::bDsFull;
      const bool soft = turn || b >= C::bStEmpty;
      const bool both = b >= C::bDOEmpty && b < C::bDOEmpty + C::kDO;  // X's dV and Y's dP have read it
      const int out = b == C::bDvEmpty || b == C::bDkEmpty ? 4 : 1;
      mbar_init(&bars[b], soft ? kSoft + (turn && C::kTurns ? 1 : 0) : both ? 2 : out);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (role == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, p.status, (uint64_t)p.spin_limit_ns};
  const int i_begin = p.dkv_off[blockIdx.x], i_end = p.dkv_off[blockIdx.x + 1];
  // Only the first K and Q tiles are asked for before dQ has ended (by the loads' warp, whose waits up to there
  // are for places that are free).  All others stand here until then, since the waits below are bounded and how
  // long dQ takes is not: where other work holds some SMs, dQ's last CTAs run a whole share behind the first.
  if (role != 2 && lane == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncwarp();

  if (role >= 4) {
    // ---------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    const int sub = warp & 3, L = sub * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    uint32_t ph = 0, tail_ph = 0;
    int loads = 0;
    for (int i = i_begin; i < i_end; ++i) {
      const PackedDkvItem it = load_item(p.dkv_items + i);
      const int per = p.causal ? it.n - it.kv : it.n;
      if (it.n * kPackedTile > it.seq_len && sub == 0) {  // rows past the end in each head's last tiles
        const int first = it.seq_len - (it.n - 1) * kPackedTile;
        for (int t = it.t0 + (per - 1 - it.t0 % per); t < it.t1; t += per) {
          const int at = loads + t - it.t0;
          mbar_wait(&bars[C::bTailDO], tail_ph, g);
          if (!warp_aborted(g)) clear_rows<D>(smem + C::oDO + at % C::kDO * C::kBytes, first, lane);
          if (lane == 0) mbar_arrive(&bars[C::bFixedDO]);
          mbar_wait(&bars[C::bTailQ], tail_ph, g);
          if (!warp_aborted(g)) clear_rows<D>(smem + C::oQ + at % C::kQ * C::kBytes, first, lane);
          if (lane == 0) mbar_arrive(&bars[C::bFixedQ]);
          tail_ph ^= 1;
        }
      }
      loads += it.t1 - it.t0;
      // dV is complete before dK, and its place is free for the next item while dK is written
      const long long row = (long long)it.row0 + L;
      float *part = p.parts + (it.slot >= 0 ? (size_t)it.slot * (2 * 128 * D) + L * D : 0);
#pragma unroll
      for (int is_k = 0; is_k < 2; ++is_k) {
        bool ok = mbar_wait(&bars[is_k ? C::bDkFull : C::bDvFull], ph, g);
        __syncwarp();
        tc_fence_after();
        ok &= L < it.rows;
        const uint32_t acc = tl + (is_k ? C::cDK : C::cDV);
        uint64_t *empty = &bars[is_k ? C::bDkEmpty : C::bDvEmpty];
        if (it.slot >= 0) {
          write_part<D>(acc, part + is_k * 128 * D, p.wide_dkv);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(empty);
          continue;
        }
        __nv_bfloat16 *to = is_k ? p.dk + row * p.dk_row + it.head * p.dk_head
                                 : p.dv + row * p.dv_row + it.head * p.dv_head;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          OutRow out;
          out.read(acc + c, is_k ? p.scale : 1.f);
          if (c + 32 == D) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty);
          }
          if (ok) out.write(to + c, p.wide_dkv);
          __syncwarp();
        }
      }
      ph ^= 1;
    }
  } else if (role >= 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    uint32_t lead = elect_one();
    auto wait = [&](int bar, uint32_t ph) {
      if (!mbar_wait(&bars[bar], ph, g)) lead = 0;
    };
    if (role == 2 && lane == 0) {
      // -------------------------------------------------------------- TMA
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmDO);
      Ring<C::kQ> rq;
      Ring<C::kDO> rd;
      Ring<C::kSt> rs;
      uint32_t e_ph = 1, nk = 0, nv = 0, nq = 0, nst = 0, ndo = 0;
      bool live = true;
      auto load = [&](int full, int empty, uint32_t ph, uint32_t at, const CUtensorMap *m, int row, int head) {
        live = live && mbar_wait(&bars[empty], ph ^ 1, g);
        if (!live) return 0u;
        mbar_arrive_expect_tx(&bars[full], C::kBytes);
        C::load(smem + at, m, &bars[full], row, head);
        return 1u;
      };
      for (int i = i_begin; i < i_end; ++i) {
        const PackedDkvItem it = load_item(p.dkv_items + i);
        const int q_first = p.causal ? it.kv : 0, per = it.n - q_first;
        int head = it.head * p.group + it.t0 / per, q = q_first + it.t0 % per;
        for (int t = it.t0; t < it.t1; ++t) {
          const int row = it.seq_row0 + q * kPackedTile;
          if (t == it.t0) nk += load(C::bKFull, C::bKEmpty, e_ph ^ 1, C::oK, &tmK, it.row0, it.head);
          nq += load(C::bQFull + rq.st, C::bQEmpty + rq.st, rq.ph, C::oQ + rq.st * C::kBytes, &tmQ, row, head);
          if (i == i_begin && t == it.t0) {  // every CTA has an item, so this grid ends behind dQ's
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("fence.proxy.async.global;" ::: "memory");
          }
          live = live && mbar_wait(&bars[C::bStEmpty + rs.st], rs.ph ^ 1, g);
          if (live) {
            mbar_arrive_expect_tx(&bars[C::bStFull + rs.st], 1024);
            bulk_load(smem + C::oSTAT + rs.st * 1024, p.stats + ((size_t)head * p.n_tiles + it.tile0 + q) * 256, 1024,
                      &bars[C::bStFull + rs.st]);
            ++nst;
          }
          if (t == it.t0) {
            nv += load(C::bVFull, C::bVEmpty, e_ph ^ 1, C::oV, &tmV, it.row0, it.head);
            e_ph ^= 1;
          }
          ndo += load(C::bDOFull + rd.st, C::bDOEmpty + rd.st, rd.ph, C::oDO + rd.st * C::kBytes, &tmDO, row, head);
          rq.next();
          rs.next();
          rd.next();
          if (++q == it.n) {
            q = q_first;
            ++head;
          }
        }
      }
      // copies still in flight land before the CTA exits
      auto drain = [&](int bar, uint32_t n, uint32_t stages) {
        for (uint32_t s = 0; s < stages; ++s) {
          const uint32_t f = n / stages + (s < n % stages ? 1u : 0u);
          if (f) mbar_drain(&bars[bar + s], (f - 1) & 1, g.limit_ns);
        }
      };
      drain(C::bKFull, nk, 1);
      drain(C::bVFull, nv, 1);
      drain(C::bQFull, nq, C::kQ);
      drain(C::bDOFull, ndo, C::kDO);
      drain(C::bStFull, nst, C::kSt);
    } else if (role == 0) {
      // ------------------------------------------------ X: dV (and S^T)
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idV = idesc_bf16(128, D, 0, 1);
      const uint64_t dk = sw128_desc(smem_u32(smem + C::oK), 16, 1024);
      const uint64_t dq0 = sw128_desc(smem_u32(smem + C::oQ), 16, 1024);
      const uint64_t ddo0 = sw128_desc(smem_u32(smem + C::oDO), C::kPanel, 1024);
      Ring<C::kQ> rq;
      Ring<C::kDO> rd;
      uint32_t k_ph = 0, p_ph = 0, o_ph = 1, fix_ph = 0, buf = 0;
      auto issue_s = [&](bool pass) {  // kTurns
        tc_fence_after();
        const uint64_t dq = dq0 + ((rq.st * C::kBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (pass && kk == D / 16 - 2 && lead) mbar_arrive(&bars[C::bDsFull]);
          mma_ss_if(lead, tmem, dk + C::kmajor(kk), dq + C::kmajor(kk), idS, kk > 0);
        }
        tc_commit_if(lead, &bars[C::bSFull]);
        rq.next();
      };
      for (int i = i_begin; i < i_end; ++i) {
        const PackedDkvItem it = load_item(p.dkv_items + i);
        const int per = p.causal ? it.n - it.kv : it.n, total = it.t1 - it.t0;
        const bool ragged = it.n * kPackedTile > it.seq_len;
        int left = per - it.t0 % per;  // Q tiles of the head from this one on
        if (C::kTurns) {
          wait(C::bKFull, k_ph);
          k_ph ^= 1;
          wait(C::bQFull + rq.st, rq.ph);
          issue_s(false);
          if (total == 1) tc_commit_if(lead, &bars[C::bKEmpty]);
        }
        for (int t = 0; t < total; ++t) {
          const bool more = t + 1 < total;
          wait(C::bDOFull + rd.st, rd.ph);
          if (ragged && left == 1) {  // the head's last tile: its rows past the end are summed over
            if (lead) mbar_arrive(&bars[C::bTailDO]);
            wait(C::bFixedDO, fix_ph);
            fix_ph ^= 1;
          }
          left = left == 1 ? per : left - 1;
          if (t == 0) {  // the item before has been written out
            wait(C::bDvEmpty, o_ph);
            o_ph ^= 1;
          }
          if (C::kTurns && more) wait(C::bQFull + rq.st, rq.ph);
          wait(C::bPFull + buf, p_ph);
          p_ph ^= (int)buf == C::kS - 1;  // the buffers' parity changes after the last one
          tc_fence_after();
          const uint64_t ddo = ddo0 + ((rd.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (C::kTurns && !more && kk == 6 && lead) mbar_arrive(&bars[C::bDsFull]);
            mma_ts_if(lead, tmem + C::cDV, tmem + buf * 128 + packed_col(kk), ddo + ((kk * 2048) >> 4), idV,
                      (t > 0 || kk > 0) ? 1u : 0u);
          }
          if (!C::kTurns) tc_commit_if(lead, &bars[C::bSEmpty + buf]);
          tc_commit_if(lead, &bars[C::bDOEmpty + rd.st]);
          if (!more) tc_commit_if(lead, &bars[C::bDvFull]);
          rd.next();
          buf = (buf + 1) % C::kS;
          if (C::kTurns && more) {
            issue_s(true);  // dV has read P: MMAs of one warp run in issue order
            if (t + 2 == total) tc_commit_if(lead, &bars[C::bKEmpty]);
          }
        }
      }
      tc_commit_if(elect_one(), &bars[C::bFinalX]);
      mbar_drain(&bars[C::bFinalX], 0, g.limit_ns);
    } else if (role == 1) {
      // ----------------------------------------------- Y: dP^T and dK
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idK = idesc_bf16(128, D, 0, 1);
      const uint64_t dv = sw128_desc(smem_u32(smem + C::oV), 16, 1024);
      const uint64_t ddo0 = sw128_desc(smem_u32(smem + C::oDO), 16, 1024);
      const uint64_t dq0 = sw128_desc(smem_u32(smem + C::oQ), C::kPanel, 1024);
      Ring<C::kQ> rq;
      Ring<C::kDO> rd;
      uint32_t v_ph = 0, ds_ph = 0, o_ph = 1, fix_ph = 0;
      auto issue_dp = [&](bool last) {
        const uint64_t ddo = ddo0 + ((rd.st * C::kBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (C::kTurns && kk == D / 16 - 2 && lead) mbar_arrive(&bars[C::bPFull]);
          mma_ss_if(lead, tmem + C::cDP, dv + C::kmajor(kk), ddo + C::kmajor(kk), idS, kk > 0);
        }
        tc_commit_if(lead, &bars[C::bDpFull]);
        tc_commit_if(lead, &bars[C::bDOEmpty + rd.st]);
        if (last) tc_commit_if(lead, &bars[C::bVEmpty]);
        rd.next();
      };
      for (int i = i_begin; i < i_end; ++i) {
        const PackedDkvItem it = load_item(p.dkv_items + i);
        const int per = p.causal ? it.n - it.kv : it.n, total = it.t1 - it.t0;
        const bool ragged = it.n * kPackedTile > it.seq_len;
        wait(C::bVFull, v_ph);
        v_ph ^= 1;
        wait(C::bDOFull + rd.st, rd.ph);
        tc_fence_after();
        issue_dp(total == 1);
        int left = per - it.t0 % per;
        for (int t = 0; t < total; ++t) {
          const bool more = t + 1 < total;
          if (more) wait(C::bDOFull + rd.st, rd.ph);
          wait(C::bQFull + rq.st, rq.ph);
          if (ragged && left == 1) {
            if (lead) mbar_arrive(&bars[C::bTailQ]);
            wait(C::bFixedQ, fix_ph);
            fix_ph ^= 1;
          }
          left = left == 1 ? per : left - 1;
          if (t == 0) {
            wait(C::bDkEmpty, o_ph);
            o_ph ^= 1;
          }
          wait(C::bDsFull, ds_ph);
          ds_ph ^= 1;
          tc_fence_after();
          const uint64_t dq = dq0 + ((rq.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_if(lead, tmem + C::cDK, tmem + C::cDP + packed_col(kk), dq + ((kk * 2048) >> 4), idK,
                      (t > 0 || kk > 0) ? 1u : 0u);
          tc_commit_if(lead, &bars[C::bQEmpty + rq.st]);
          rq.next();
          if (more)
            issue_dp(t + 2 == total);  // dK has read dS
          else
            tc_commit_if(lead, &bars[C::bDkFull]);
        }
      }
      tc_commit_if(elect_one(), &bars[C::bFinalY]);
      mbar_drain(&bars[C::bFinalY], 0, g.limit_ns);
    } else if (role == 3 && !C::kTurns) {
      // -------------------------------------------------------- Z: S^T
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      const uint64_t dk = sw128_desc(smem_u32(smem + C::oK), 16, 1024);
      const uint64_t dq0 = sw128_desc(smem_u32(smem + C::oQ), 16, 1024);
      Ring<C::kQ> rq;
      uint32_t k_ph = 0, e_ph = 1, buf = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const PackedDkvItem it = load_item(p.dkv_items + i);
        const int total = it.t1 - it.t0;
        wait(C::bKFull, k_ph);
        k_ph ^= 1;
        for (int t = 0; t < total; ++t) {
          wait(C::bQFull + rq.st, rq.ph);
          wait(C::bSEmpty + buf, e_ph);
          e_ph ^= (int)buf == C::kS - 1;
          tc_fence_after();
          const uint64_t dq = dq0 + ((rq.st * C::kBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_if(lead, tmem + buf * 128, dk + C::kmajor(kk), dq + C::kmajor(kk), idS, kk > 0);
          tc_commit_if(lead, &bars[C::bSFull + buf]);
          rq.next();
          buf = (buf + 1) % C::kS;
        }
        tc_commit_if(lead, &bars[C::bKEmpty]);
      }
      tc_commit_if(elect_one(), &bars[C::bFinalZ]);
      mbar_drain(&bars[C::bFinalZ], 0, g.limit_ns);
    }
  } else {
    // -------------------------------------------------------- P and dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int sub = warp & 3, c0 = (warp >> 2) * kCols;  // its columns of S^T and dP^T
    const int before = sub * 32 + lane - c0;  // of its columns, those ahead of its KV row
    const uint8_t *stats = smem + C::oSTAT + c0 * 4;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16) + c0, tP = tl + C::cDP;
    const uint64_t sc2 = dup2(p.scale_log2);
    Ring<C::kSt> rs;
    uint32_t s_ph = 0, dp_ph = 0, buf = 0;
    for (int i = i_begin; i < i_end; ++i) {
      const PackedDkvItem it = load_item(p.dkv_items + i);
      const int per = p.causal ? it.n - it.kv : it.n, total = it.t1 - it.t0;
      int k = it.t0 % per;
      const int last = it.seq_len - (it.n - 1) * kPackedTile - c0;
      for (int t = 0; t < total; ++t) {
        // a causal KV tile's first Q tile of each head is on the diagonal
        const bool diagonal = p.causal && k == 0;
        k = k + 1 == per ? 0 : k + 1;
        // those inside the sequence: fewer in the head's last tile only
        const int cols = k == 0 ? last : kCols;
        const ulonglong2 *nl = reinterpret_cast<const ulonglong2 *>(stats + rs.st * 1024);
        const ulonglong2 *nd = nl + 32;
        mbar_wait(&bars[C::bStFull + rs.st], rs.ph, g);
        mbar_wait(&bars[C::bSFull + buf], s_ph, g);
        const uint32_t tS = tl + buf * 128, p_bar = C::bPFull + buf;
        buf = (buf + 1) % C::kS;
        s_ph ^= buf == 0;
        __syncwarp();
        tc_fence_after();
        uint32_t x[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) tmem_ld32_nowait(tS + 32 * c, x[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) reg_order32(x[c]);
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 l4 = nl[8 * c + (e >> 2)];
            float a, b, u, v;
            unpack2(fma2(pack2(x[c][e], x[c][e + 1]), sc2, l4.x), a, b);
            unpack2(fma2(pack2(x[c][e + 2], x[c][e + 3]), sc2, l4.y), u, v);
            x[c][e] = __float_as_uint(ex2(a));
            x[c][e + 1] = __float_as_uint(ex2(b));
            x[c][e + 2] = __float_as_uint(ex2(u));
            x[c][e + 3] = __float_as_uint(ex2(v));
          }
        if (diagonal) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e < before) x[c][e] = 0u;
        }
        if (cols < kCols) {  // replaced, as dS below: what Q and dO hold there may not be finite
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= cols) x[c][e] = 0u;
        }
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            pk[e >> 1] = pack_bf16(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
          tmem_st16(tS + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[p_bar]);

        mbar_wait(&bars[C::bDpFull], dp_ph, g);
        dp_ph ^= 1;
        __syncwarp();
        tc_fence_after();
        uint32_t y[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) tmem_ld32_nowait(tP + 32 * c, y[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) reg_order32(y[c]);
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 d4 = nd[8 * c + (e >> 2)];
            float a, b, u, v;
            unpack2(mul2(pack2(x[c][e], x[c][e + 1]), add2(pack2(y[c][e], y[c][e + 1]), d4.x)), a, b);
            unpack2(mul2(pack2(x[c][e + 2], x[c][e + 3]), add2(pack2(y[c][e + 2], y[c][e + 3]), d4.y)), u, v);
            pk[e >> 1] = pack_bf16(a, b);
            pk[(e >> 1) + 1] = pack_bf16(u, v);
          }
          if (cols < kCols) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              if (32 * c + e >= cols) pk[e >> 1] = 0u;
              else if (32 * c + e + 1 >= cols) pk[e >> 1] &= 0xffffu;
            }
          }
          tmem_st16(tP + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[C::bDsFull]);
          mbar_arrive(&bars[C::bStEmpty + rs.st]);
        }
        rs.next();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (role == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the parts of a KV tile's dK and dV in their order.  Bound by the bytes
// of the parts, which mostly come from L2.
template <int D>
__global__ void __launch_bounds__(256) dash_packed_sum(const PackedBwdParams p) {
  const PackedSum it = load_item(p.sums + blockIdx.x);
  const bool is_k = blockIdx.y != 0;
  const float *src = p.parts + (size_t)it.slot * (2 * 128 * D) + (is_k ? 128 * D : 0);
  __nv_bfloat16 *out = is_k ? p.dk + it.row0 * p.dk_row + it.head * p.dk_head
                            : p.dv + it.row0 * p.dv_row + it.head * p.dv_head;
  const long long row_stride = is_k ? p.dk_row : p.dv_row;
  const float scale = is_k ? p.scale : 1.f;
  // blockIdx.z takes a quarter of the rows
  for (int x = threadIdx.x; x < 32 * D / 4; x += 256) {
    const int r = blockIdx.z * 32 + x / (D / 4), c = x % (D / 4) * 4;
    if (r >= it.rows) break;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < it.n; ++k) {
      const float4 v = *reinterpret_cast<const float4 *>(src + (size_t)k * (2 * 128 * D) + r * D + c);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    *reinterpret_cast<uint2 *>(out + r * row_stride + c) =
        make_uint2(pack_bf16(scale * sum.x, scale * sum.y), pack_bf16(scale * sum.z, scale * sum.w));
  }
}

template <class Cfg>
constexpr int smem_bytes() {
  return Cfg::kSmem > (uint32_t)kMinSmemOneCtaPerSm ? (int)Cfg::kSmem : kMinSmemOneCtaPerSm;
}

template <class K>
cudaError_t prepare_kernel(K kernel, int smem, int regs) {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;  // the register split counts on it
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int D>
cudaError_t prepare_t() {
  cudaError_t e = prepare_kernel(dash_packed_dq_kernel<D>, smem_bytes<DqCfg<D>>(), kRegsLaunch);
  return e == cudaSuccess ? prepare_kernel(dash_packed_dkv_kernel<D>, smem_bytes<DkvCfg<D>>(), kRegsLaunch) : e;
}

template <int D>
cudaError_t launch_t(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const CUtensorMap &dout,
                     const PackedBwdParams &p, int dq_ctas, int dkv_ctas, cudaStream_t stream) {
  cudaError_t e =
      launch(dash_packed_dq_kernel<D>, dq_ctas, kThreads, smem_bytes<DqCfg<D>>(), stream, nullptr, q, k, v, dout, p);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = overlap_attr();
  e = launch(dash_packed_dkv_kernel<D>, dkv_ctas, kThreads, smem_bytes<DkvCfg<D>>(), stream, &attr, q, k, v, dout, p);
  if (e != cudaSuccess || !p.n_sums) return e;
  return launch(dash_packed_sum<D>, dim3(p.n_sums, 2, 4), 256, 0, stream, nullptr, p);
}

}  // namespace

cudaError_t prepare_packed_bwd(int D) { return D == 64 ? prepare_t<64>() : prepare_t<128>(); }

cudaError_t launch_packed_bwd(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const CUtensorMap &dout, const PackedBwdParams &p, int dq_ctas, int dkv_ctas,
                              cudaStream_t stream) {
  return D == 64 ? launch_t<64>(q, k, v, dout, p, dq_ctas, dkv_ctas, stream)
                 : launch_t<128>(q, k, v, dout, p, dq_ctas, dkv_ctas, stream);
}

}  // namespace dash
