// Packed, grouped-head softmax attention forward for sm_103a.
//
// One pass over the keys with the running maximum and sum of the softmax:
//   m' = max(m, max_j x_j),  l' = l 2^(m-m') + sum_j 2^(x_j - m'),
//   O' = O 2^(m-m') + P V,   x = scale log2(e) q.k,  P = 2^(x - m'),
// O / l at the end and LSE = ln2 (m + log2 l).  O stays in tensor memory.  The
// maximum a row refers to moves only when it has grown by more than 2^8
// (kLazy): until then P may exceed 1, which costs no precision (P keeps its
// eight bits, l and O are fp32), and the rescaling of O, a round trip through
// registers, happens a few times a row at most.
//
// A persistent CTA walks the items that the plan gave it.  An item is two
// 128-row Q tiles on one K/V head, so that every K and V tile in shared memory
// feeds four MMAs and one tile's softmax runs under the other tile's MMAs:
//   tensor pipe   PV0(j) S0(j+1) | PV1(j) S1(j+1) | PV0(j+1) ...
//   softmax 0              ......| S0(j+1) -> P0  |
// Two heads of a group on the same rows share keys exactly; with one head per
// group (or an odd one left over) two neighbouring tiles of a head pair up.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1 (a thread owns a row), 12-15
// the epilogue, 8 and 11 MMA issue for tile 0 and 1, 9 TMA, 10 clears the V rows past
// the sequence's end in the last KV tile (they belong to the next sequence or to nobody: P is 0
// there, but 0 x NaN is NaN).  K rows past the end are masked after the
// product, Q rows past the end are computed and not written.
//
// Tensor memory: S0 at 0, S1 at 128, O0 at 256, O1 at 256+D; P, packed bf16 and
// rounded once as the MMA's operand, overwrites the first half of its S.  At
// D = 64 there is room for P beside S (at 384 and 448): the next score then runs
// as soon as this one is in registers, so that the softmax, which takes longer
// than the products there, never waits for them (16 heads of 4096 tokens:
// 707 TFLOPS against 670).
#include <cuda_runtime.h>

#include "packed.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128;   // 512 threads x 128 registers
constexpr int kRegsSoftmax = 176;  // a row of S in registers
constexpr int kRegsOther = 88;
constexpr int kRegsOut = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * (kRegsOther + kRegsOut) <= kRegsLaunch * kThreads,
              "register split exceeds the CTA's allocation");
constexpr float kLazy = 8.f;       // log2 growth of a row's maximum that is left standing

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr int kStages = D == 128 ? 5 : 8;  // K and V tiles in turn
  static constexpr uint32_t oQ = 0;                 // two Q tiles
  static constexpr uint32_t oKV = 2 * kTile;
  static constexpr uint32_t oBAR = oKV + kStages * kTile;
  static constexpr int kNumBars = 25 + 2 * kStages;
  static constexpr uint32_t oMISC = oBAR + kNumBars * 8;
  static constexpr uint32_t oSTAT = oMISC + 16;     // {maximum, sum} of each tile's rows
  static constexpr uint32_t kSmemBytes = oSTAT + 2 * 128 * 8;
  static constexpr uint32_t cO = 256;
  static constexpr bool kApart = D == 64;  // P beside S
  static __device__ __forceinline__ constexpr uint32_t cP(int s) { return kApart ? 384 + 64 * s : 128 * s; }
};
static_assert(Cfg<128>::kSmemBytes <= 232448 && Cfg<64>::kSmemBytes <= 232448, "shared memory of one CTA");

enum {
  bQFull = 0, bQEmpty = 2, bSFull = 4, bOFull = 6, bFinal = 8, bVTail = 10, bPFull = 11, bLFull = 13, bOEmpty = 15,
  bSRead = 17, bPvDone = 19, bVFixed = 21, bKvFull0 = 25
};
// Cleared V tails that one MMA warp may be ahead of the other by: an item holds
// at least two stages of the ring until both have read it.
constexpr int kFixed = 4;
static_assert(Cfg<128>::kStages <= 2 * kFixed && Cfg<64>::kStages <= 2 * kFixed && bVFixed + kFixed == bKvFull0,
              "a warp could miss a cleared tail");

__device__ __forceinline__ PackedFwdItem load_item(const PackedFwdItem *p) {
  PackedFwdItem it;
  const int4 *s = reinterpret_cast<const int4 *>(p);
  int4 *d = reinterpret_cast<int4 *>(&it);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = __ldg(s + i);
  return it;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
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

// Ring position: stage and the parity of its current pass.
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dash_packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const PackedFwdParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = warp_id(), lane = threadIdx.x & 31;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::oBAR);
  uint64_t *kvFull = bars + bKvFull0, *kvEmpty = kvFull + C::kStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::oMISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::oMISC + 4);

  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemMisaligned);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[bQFull + s], 1);
      mbar_init(&bars[bQEmpty + s], 1);
      mbar_init(&bars[bSFull + s], 1);
      mbar_init(&bars[bPFull + s], C::kApart ? 4 : 5);  // four softmax warps and the turn
      mbar_init(&bars[bSRead + s], 4);
      mbar_init(&bars[bPvDone + s], 1);
      mbar_init(&bars[bLFull + s], 4);
      mbar_init(&bars[bOEmpty + s], 4);
      mbar_init(&bars[bOFull + s], 1);
      mbar_init(&bars[bFinal + s], 1);
    }
    for (int k = 0; k < kFixed; ++k) mbar_init(&bars[bVFixed + k], 1);
    mbar_init(&bars[bVTail], 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&kvFull[s], 1);
      mbar_init(&kvEmpty[s], 2);  // both MMA warps
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, p.status, (uint64_t)p.spin_limit_ns};
  float2 *stat = reinterpret_cast<float2 *>(smem + C::oSTAT);
  const int i_begin = p.cta_off[blockIdx.x], i_end = p.cta_off[blockIdx.x + 1];

  if (warp >= 12) {
    // ---------------------------------------------------------- epilogue
    // The two tiles' O in turn, while the softmax warps are at the next item.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    const int sub = warp & 3, L = sub * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    uint32_t ph[2] = {0, 0};
    for (int i = i_begin; i < i_end; ++i) {
      const PackedFwdItem it = load_item(p.items + i);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (it.nkv[s] == 0) continue;
        bool ok = mbar_wait(&bars[bLFull + s], ph[s], g);
        ok &= mbar_wait(&bars[bOFull + s], ph[s], g);
        ph[s] ^= 1;
        __syncwarp();
        tc_fence_after();
        const float2 ml = stat[s * 128 + L];
        const float inv = ml.y > 0.f ? 1.f / ml.y : 0.f;
        ok &= L < it.rows[s];
        const long long row = (long long)it.row0[s] + L;
        __nv_bfloat16 *orow = p.o + row * p.o_row + it.head[s] * p.o_head;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tl + C::cO + s * D + c0, r);
          if (ok) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t *a = r + 16 * k + 2 * e;
                w[e] = pack_bf16(inv * __uint_as_float(a[0]), inv * __uint_as_float(a[1]));
              }
              st_32b(orow + c0 + 16 * k, w, p.wide);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[bOEmpty + s]);
        if (ok) p.lse[it.head[s] * p.lse_head + row] = (ml.x + log2f(ml.y)) * 0.6931471805599453f;
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 9 && lane == 0) {
      // -------------------------------------------------------------- TMA
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      Ring<C::kStages> r;
      uint32_t q_ph[2] = {1, 1};     // parity to wait for on the empty barriers: the first pass is free
      uint32_t q_fills[2] = {0, 0};
      uint32_t fills = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const PackedFwdItem it = load_item(p.items + i);
        const int n = max(it.nkv[0], it.nkv[1]);
        auto load_q = [&](int s, int row0, int head) {
          mbar_wait(&bars[bQEmpty + s], q_ph[s], g);
          q_ph[s] ^= 1;
          if (*g.abort) return;
          mbar_arrive_expect_tx(&bars[bQFull + s], C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::oQ + s * C::kTile + pn * C::kPanel, &tmQ, &bars[bQFull + s], pn * 64, row0,
                        head);
          ++q_fills[s];
        };
        auto load_kv = [&](const CUtensorMap *m, int j) {
          mbar_wait(&kvEmpty[r.st], r.ph ^ 1, g);
          if (*g.abort) return;
          mbar_arrive_expect_tx(&kvFull[r.st], C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::oKV + r.st * C::kTile + pn * C::kPanel, m, &kvFull[r.st], pn * 64,
                        it.kv_row0 + j * kPackedTile, it.kv_head);
          ++fills;
          r.next();
        };
        load_q(0, it.row0[0], it.head[0]);
        load_kv(&tmK, 0);
        if (it.nkv[1] > 0) load_q(1, it.row0[1], it.head[1]);
        for (int j = 0; j < n; ++j) {
          load_kv(&tmV, j);
          if (j + 1 < n) load_kv(&tmK, j + 1);
        }
      }
      // copies still in flight land before the CTA exits
      for (int s = 0; s < 2; ++s)
        if (q_fills[s]) mbar_drain(&bars[bQFull + s], (q_fills[s] - 1) & 1, g.limit_ns);
      for (int s = 0; s < C::kStages; ++s) {
        const uint32_t f = fills / C::kStages + ((uint32_t)s < fills % C::kStages ? 1u : 0u);
        if (f) mbar_drain(&kvFull[s], (f - 1) & 1, g.limit_ns);
      }
    } else if (warp == 8 || warp == 11) {
      // ----------------------- MMA: a warp for each of the two Q tiles
      // One warp for both leaves the tensor pipe idle at each of its waits (a
      // wait queues behind the MMAs just issued, and answers about 100 clocks
      // later).  The warps take turns, tile 0's PV and next S, then tile 1's, so
      // that one tile's softmax runs under the other's MMAs; free running, the
      // two fall into step and softmax and MMAs take place one after the other.
      // (With P apart the softmax sets the pace and there are no turns.)
      const int s = warp == 8 ? 0 : 1;
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
      Ring<C::kStages> rk;              // next K or V tile to be read
      uint32_t q_ph = 0, p_ph = 0, o_ph = 1, r_ph = 1, fixes = 0;
      bool owed = false;                // the other warp passes the turn to this one's next P
      uint32_t lead = elect_one();      // 0 in every lane once a wait has failed: nothing more is issued
      const uint64_t dq = sw128_desc(smem_u32(smem + C::oQ + s * C::kTile), 16, 1024);
      const uint64_t dk0 = sw128_desc(smem_u32(smem + C::oKV), 16, 1024);
      const uint64_t dv0 = sw128_desc(smem_u32(smem + C::oKV), C::kPanel, 1024);
      const uint32_t tS = tmem + s * 128, tP = tmem + C::cP(s), tO = tmem + C::cO + s * D;
      auto wait = [&](int bar, uint32_t ph) {
        if (!mbar_wait(&bars[bar], ph, g)) lead = 0;
      };
      // Passing the turn is an arrival on the barrier that also counts the other
      // tile's P, so that one wait answers for both.
      auto give_turn = [&](int to) {
        if (lead) mbar_arrive(&bars[bPFull + to]);
      };
      auto issue_s = [&](int stage, bool pass) {
        if (C::kApart) {
          wait(bSRead + s, r_ph);  // the S before is in registers
          r_ph ^= 1;
        }
        tc_fence_after();
        const uint64_t dk = dk0 + ((stage * C::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4;
          if (pass && kk == D / 16 - 2) give_turn(s ^ 1);  // the other warp wakes up under the last MMAs
          mma_ss_if(lead, tS, dq + off, dk + off, idS, kk > 0);
        }
        tc_commit_if(lead, &bars[bSFull + s]);
      };
      for (int i = i_begin; i < i_end; ++i) {
        const PackedFwdItem it = load_item(p.items + i);
        const int n = max(it.nkv[0], it.nkv[1]), mine = s ? it.nkv[1] : it.nkv[0];
        const int both = min(it.nkv[0], it.nkv[1]);  // KV tiles with a turn: those of both tiles
        const bool fix = n * kPackedTile > it.kv_len;
        wait(bKvFull0 + rk.st, rk.ph);
        if (mine > 0) {  // S of the first KV tile
          wait(bQFull + s, q_ph);
          q_ph ^= 1;
          issue_s(rk.st, false);
          if (mine == 1) tc_commit_if(lead, &bars[bQEmpty + s]);
        }
        tc_commit_if(lead, &kvEmpty[rk.st]);
        rk.next();
        for (int j = 0; j < n; ++j) {
          const Ring<C::kStages> rv = rk;  // V tile j; the next K tile follows it in the ring
          rk.next();
          wait(bKvFull0 + rv.st, rv.ph);
          if (fix && j == n - 1) {
            if (lead && s == 0) mbar_arrive(&bars[bVTail]);  // it has landed: its rows past the end may be cleared
            wait(bVFixed + fixes % kFixed, fixes / kFixed & 1);
            ++fixes;
          }
          if (j + 1 < n) wait(bKvFull0 + rk.st, rk.ph);
          const uint64_t dv = dv0 + ((rv.st * C::kTile) >> 4);
          if (j < mine) {
            if (j == 0) {
              wait(bOEmpty + s, o_ph);
              o_ph ^= 1;
            }
            const bool more = j + 1 < mine;
            if (C::kApart && more) issue_s(rk.st, false);
            // P stands in tensor memory, O is at its scale, and the turn has come: tile 1's from tile 0's warp at the
            // same KV tile, tile 0's from tile 1's warp at the KV tile before, or, where tile 1 had none, from itself.
            // So no turn is passed to a warp before it has taken its last one.  (Tile 1 never has more KV tiles.)
            const bool pass = !C::kApart && j < both;
            if (!C::kApart && s == 0 && !owed) give_turn(0);
            owed = pass;
            wait(bPFull + s, p_ph);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts_if(lead, tO, tP + kk * 8, dv + ((kk * 2048) >> 4), idO, (j > 0 || kk > 0) ? 1u : 0u);
            p_ph ^= 1;
            if (C::kApart) tc_commit_if(lead, &bars[bPvDone + s]);
            if (more) {
              if (!C::kApart) issue_s(rk.st, pass);  // MMAs run in issue order: PV has read P before S overwrites it
              if (j + 2 == mine) tc_commit_if(lead, &bars[bQEmpty + s]);
            } else {
              if (pass) give_turn(s ^ 1);
              tc_commit_if(lead, &bars[bOFull + s]);
            }
          }
          // each tile is free when both warps' MMAs have read it (a warp that has none arrives at once)
          tc_commit_if(lead, &kvEmpty[rv.st]);
          if (j + 1 < n) {
            tc_commit_if(lead, &kvEmpty[rk.st]);
            rk.next();
          }
        }
      }
      // every MMA has completed before tensor memory is released (at once if none was issued)
      tc_commit_if(elect_one(), &bars[bFinal + s]);
      mbar_drain(&bars[bFinal + s], 0, g.limit_ns);
    } else if (warp == 10) {
      // ------------------------------- V rows past the end of the sequence
      uint32_t loads = 0, tail_ph = 0, fixes = 0;
      for (int i = i_begin; i < i_end; ++i) {
        const PackedFwdItem it = load_item(p.items + i);
        const int n = max(it.nkv[0], it.nkv[1]);
        loads += 2 * n;  // the item's last V tile is its last load
        if (n * kPackedTile > it.kv_len) {
          mbar_wait(&bars[bVTail], tail_ph, g);
          tail_ph ^= 1;
          uint8_t *v = smem + C::oKV + (loads - 1) % C::kStages * C::kTile;
          const int first = it.kv_len - (n - 1) * kPackedTile;
          if (!warp_aborted(g)) {
            // a row is 128 bytes of each panel, whatever the swizzle does inside it
            for (int x = first * 8 + lane; x < kPackedTile * 8; x += 32)
#pragma unroll
              for (int pn = 0; pn < C::kPanels; ++pn)
                *reinterpret_cast<uint4 *>(v + pn * C::kPanel + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[bVFixed + fixes % kFixed]);
          ++fixes;
        }
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int s = warp >> 2, sub = warp & 3;
    const int L = sub * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    const uint32_t tS = tl + s * 128, tP = tl + C::cP(s), tO = tl + C::cO + s * D;
    uint32_t s_ph = 0, o_ph = 0, v_ph = 0;
    for (int i = i_begin; i < i_end; ++i) {
      const PackedFwdItem it = load_item(p.items + i);
      const int n = s ? it.nkv[1] : it.nkv[0];
      if (n == 0) continue;
      const int q_pos = (s ? it.q0[1] : it.q0[0]) + L;
      // keys this row attends: those of the sequence, up to its own position
      const int limit = p.causal ? min(it.kv_len, q_pos + 1) : it.kv_len;
      float m = -INFINITY;   // the maximum the row refers to (scaled, log2)
      uint64_t l2 = 0;       // its sum, in two halves
      // After an abort the loop runs on with whatever tensor memory holds: no
      // wait blocks any more, and the status word tells that O is not valid.
      for (int j = 0; j < n; ++j) {
        mbar_wait(&bars[bSFull + s], s_ph, g);
        s_ph ^= 1;
        __syncwarp();
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_nowait(tS + 32 * c, x[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_order32(x[c]);
        if (C::kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[bSRead + s]);
        }
        const int cols = limit - j * kPackedTile;  // valid columns of this tile
        if (__any_sync(0xffffffffu, cols < kPackedTile)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= cols) x[c][e] = 0xff800000u;  // -inf
        }
        float mx[4];  // four chains side by side
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(x[c][e])), __uint_as_float(x[c][e + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        if (C::kApart && j > 0) {  // the last PV has read P
          mbar_wait(&bars[bPvDone + s], v_ph, g);
          v_ph ^= 1;
          __syncwarp();
          tc_fence_after();
        }
        if (j == 0) {
          m = top == -INFINITY ? 0.f : top;
        } else if (__any_sync(0xffffffffu, top > m + kLazy)) {
          // PV(j-1) is complete (with P in S's place it completed before S(j) did), so O may be rewritten here.
          // The vote decides whether the warp does, each row for itself whether it moves (else its factor is 1):
          // its bits do not depend on the warp's other rows, which may belong to another sequence or to nobody.
          const float m_new = top > m + kLazy ? top : m;
          const float f = ex2(m - m_new);
          m = m_new;
          const uint64_t f2 = pack2(f, f);
          l2 = mul2(l2, f2);
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t r[16];
            tmem_ld16(tO + c0, r);
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st16(tO + c0, r);
          }
        }
        const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), nm2 = pack2(-m, -m);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t y2 = fma2(pack2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sc2, nm2);
            float a, b;
            unpack2(y2, a, b);
            a = ex2(a);
            b = ex2(b);
            x[c][e] = __float_as_uint(a);
            x[c][e + 1] = __float_as_uint(b);
            pk[e >> 1] = pack_bf16(a, b);
          }
          tmem_st16(tP + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[bPFull + s]);
        // the sum is not on the product's path
        uint64_t acc2[4] = {l2, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 32; e += 2)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc2[c] = add2(acc2[c], pack2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])));
        l2 = add2(add2(acc2[0], acc2[1]), add2(acc2[2], acc2[3]));
      }
      // The last product's completion also says that the item before has been
      // written out (the product waited for it), so its row of `stat` is free.
      mbar_wait(&bars[(C::kApart ? bPvDone : bOFull) + s], C::kApart ? v_ph : o_ph, g);
      o_ph ^= 1;
      v_ph ^= 1;
      float la, lb;
      unpack2(l2, la, lb);
      stat[s * 128 + L] = make_float2(m, la + lb);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bLFull + s]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
int smem_bytes() {
  return Cfg<D>::kSmemBytes > (uint32_t)kMinSmemOneCtaPerSm ? (int)Cfg<D>::kSmemBytes : kMinSmemOneCtaPerSm;
}

template <int D>
cudaError_t prepare_t() {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, dash_packed_fwd_kernel<D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
  return cudaFuncSetAttribute(dash_packed_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<D>());
}

}  // namespace

cudaError_t prepare_packed_fwd(int D) { return D == 64 ? prepare_t<64>() : prepare_t<128>(); }

cudaError_t launch_packed_fwd(int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const PackedFwdParams &p, int num_ctas, cudaStream_t stream) {
  return D == 64 ? launch(dash_packed_fwd_kernel<64>, num_ctas, kThreads, smem_bytes<64>(), stream, nullptr, q, k, v, p)
                 : launch(dash_packed_fwd_kernel<128>, num_ctas, kThreads, smem_bytes<128>(), stream, nullptr, q, k, v, p);
}

}  // namespace dash
