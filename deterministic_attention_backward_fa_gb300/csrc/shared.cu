// Decode attention over a prefix that all sequences of a batch share, computed
// once for all.  The rows (sequence, Q head) of a K/V head's group form one
// matrix: B x group rows attend the same tokens, which is attention of many
// queries on one key sequence, so the tensor cores take it and K and V are read
// once per 256 rows.  Each CTA has (split of the prefix, up to two tiles of 128
// rows, K/V head) and leaves per row its softmax average with maximum and sum,
// as a split of dash_decode_kernel does; that kernel attends the tokens behind
// the prefix, and the same join adds all parts.
//
// Per row one pass over the split's KV tiles of 128 tokens:
//   m' = max(m, max_j x_j),  l' = l 2^(m-m') + sum_j 2^(x_j - m'),
//   O' = O 2^(m-m') + P V,   x = scale log2(e) q.k,  P = 2^(x - m'),
// with S, P (bf16, in S's place) and O in tensor memory.  The maximum moves when
// it has grown by 2^8 (kLazy), or from nothing.
// A sequence may end inside the prefix.  What it does not attend has P = 0, and
// V as the other rows attend it: 0 times a NaN or an infinity is then a NaN, and
// the join makes such a row anew, from the tokens that the sequence has (paged.cu).
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1 (a thread owns a row), 8 and 9 MMA
// issue for tile 0 and 1, 12-15 fetch K and V: a token's row lies wherever its
// page does, so rows are fetched with 16-byte asynchronous copies (16 lanes a
// row at D = 128) into the swizzled layout that the MMAs read.  A copy's end
// arrives on its stage's barrier by itself; the MMA warps put the proxy fence
// between that and their reads.  (Handed over by the fetching warps, which wait
// for one load after they have issued another, a stage comes late.)
//
// Bound by the products (4 D a token and row) and the bytes (4 D a token and K/V
// head), which are about even at 256 rows: 32000 tokens, 64 sequences of 4 heads
// on each of 8 K/V heads of 128 in 32 us, 18 and 19 of them those two.  What is
// left is each tile's chain of scores, softmax and product, of which two run in
// turn.  With tails of 512 tokens the call takes 69.5 us (55 with D = 64).
#include <cuda_runtime.h>

#include "packed.h"
#include "shared.h"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128;   // 512 threads x 128 registers
constexpr int kRegsSoftmax = 176;  // a row of S in registers
constexpr int kRegsOther = 80;
static_assert(2 * 128 * kRegsSoftmax + 2 * 128 * kRegsOther <= kRegsLaunch * kThreads,
              "register split exceeds the CTA's allocation");
constexpr float kLazy = 8.f;
constexpr int kMasks = 4;  // tiles whose masks are held
constexpr int kPages = 4;  // tiles whose pages are looked up ahead

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr int kStages = 5;  // K and V tiles in turn
  static constexpr uint32_t oQ = 0;  // two Q tiles
  static constexpr uint32_t oKV = 2 * kTile;
  static constexpr uint32_t oBAR = oKV + kStages * kTile;
  static constexpr int kNumBars = 8 + kMasks + 2 * kStages;
  static constexpr uint32_t oMISC = oBAR + kNumBars * 8;
  static constexpr uint32_t oMASK = oMISC + 16;
  static constexpr uint32_t kSmemBytes = oMASK + kMasks * 16;
  static constexpr uint32_t cO = 256;
};
static_assert(Cfg<128>::kSmemBytes <= 232448, "shared memory of one CTA");
enum { bSFull = 0, bPFull = 2, bOFull = 4, bFinal = 6, bMask = 8, bKvFull0 = 8 + kMasks };

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: fills with zeros, reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives on `bar` when this thread's copies so far have landed; the barrier counts it like any arrival.
__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

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
__global__ void __launch_bounds__(kThreads, 1) dash_prefix_kernel(const __grid_constant__ SharedParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = warp_id(), lane = threadIdx.x & 31;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::oBAR);
  uint64_t *kvFull = bars + bKvFull0, *kvEmpty = kvFull + C::kStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::oMISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::oMISC + 4);
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + C::oMASK);  // [kMasks][4]: tokens that count

  // the tails' kernel may start where there is room: it needs nothing of this one's
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int split = blockIdx.x, hk = blockIdx.z;
  const int rows = p.B * p.group, row0 = blockIdx.y * 2 * kPackedTile;
  const int tiles = rows - row0 > kPackedTile ? 2 : 1;  // Q tiles
  const int j0 = split * p.tiles_per_split, n = min(p.tiles_per_split, p.prefix_tiles - j0);

  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemMisaligned);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[bSFull + s], 1);
      mbar_init(&bars[bPFull + s], 5);  // four softmax warps and the turn
      mbar_init(&bars[bOFull + s], 1);
      mbar_init(&bars[bFinal + s], 1);
    }
    for (int i = 0; i < kMasks; ++i) mbar_init(&bars[bMask + i], 4);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&kvFull[s], 128);     // the fetching threads
      mbar_init(&kvEmpty[s], tiles);  // the MMA warps
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

  if (warp >= 12) {
    // -------------------------------------------------------------- loads
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    const int w = warp - 12;
    constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;  // 16-byte pieces of a row, rows of a warp's copy
    const int c = lane % kChunks, rsub = lane / kChunks;
    const uint32_t col = (uint32_t)(c >> 3) * C::kPanel;
    const int *table = p.table;  // the prefix's pages are those of the first sequence
    auto page_of = [&](int j) -> int {
      const int t = (j0 + j) * kPackedTile + w * 32 + lane;
      return j < n && t < p.first ? table[t / p.page_size] : -1;
    };
    // the pages of the next tiles, asked for side by side: each look-up takes as long as a tile's products
    int pages[kPages];
#pragma unroll
    for (int i = 0; i < kPages; ++i) pages[i] = page_of(i);
    // Q, with the first K tile; rows past the last are zero.  Every lane knows where one row lies.
    for (int s = 0; s < tiles; ++s) {
      const int mine = row0 + s * kPackedTile + w * 32 + lane, b = mine / p.group;
      const bool real = mine < rows;
      const long long a = real ? b * p.q_batch + (hk * p.group + mine - b * p.group) * p.q_head : 0;
      const uint32_t ok = __ballot_sync(0xffffffffu, real);
#pragma unroll 4
      for (int i = 0; i < 32 / kRowsPer; ++i) {
        const int from = i * kRowsPer + rsub, r = w * 32 + from;
        cp16(smem_u32(smem + C::oQ + s * C::kTile) + col + r * 128 + (((c & 7) ^ (r & 7)) << 4),
             p.q + __shfl_sync(0xffffffffu, a, from) + 8 * c, (ok >> from) & 1u);
      }
    }
    Ring<C::kStages> r;
    for (int j = 0; j < n; ++j) {
      const int t = (j0 + j) * kPackedTile + w * 32 + lane, page = pages[0];
#pragma unroll
      for (int i = 0; i + 1 < kPages; ++i) pages[i] = pages[i + 1];
      pages[kPages - 1] = page_of(j + kPages);
      const bool ok = page >= 0 && page < p.n_pages;
      if (t < p.first && !ok) atomicCAS(p.status, 0, kStatusBadPage);
      const uint32_t valid = __ballot_sync(0xffffffffu, ok);
      const int off = t % p.page_size;
      const long long ka = ok ? page * p.ks.page + off * p.ks.token + hk * p.ks.head : 0;
      const long long va = ok ? page * p.vs.page + off * p.vs.token + hk * p.vs.head : 0;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        mbar_wait(&kvEmpty[r.st], r.ph ^ 1, g);
        __syncwarp();
        if (which == 0) {
          // the masks kMasks tiles before have been read: their P was, by the products that freed this stage
          if (lane == 0) {
            masks[(j % kMasks) * 4 + w] = valid;
            mbar_arrive(&bars[bMask + j % kMasks]);
          }
        }
        const __nv_bfloat16 *base = which ? p.v : p.k;
        const uint32_t dst = smem_u32(smem + C::oKV + r.st * C::kTile) + col;
        if (!warp_aborted(g)) {
#pragma unroll
          for (int i = 0; i < 32 / kRowsPer; ++i) {
            const int from = i * kRowsPer + rsub, rr = w * 32 + from;
            const long long a = __shfl_sync(0xffffffffu, which ? va : ka, from);
            cp16(dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), base + a + 8 * c, (valid >> from) & 1u);
          }
        }
        cp_arrive(&kvFull[r.st]);
        r.next();
      }
    }
    cp_wait_all();
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    const int s = warp - 8;
    if (s < tiles) {
      // --------------------------------------- MMA: a warp for each Q tile
      // They take turns, as in the packed forward: tile 0's PV and next S, then tile
      // 1's, so that one tile's softmax runs under the other's MMAs.
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
      Ring<C::kStages> rk;          // next K or V tile to be read
      uint32_t p_ph = 0;
      uint32_t lead = elect_one();  // 0 in every lane once a wait has failed: nothing more is issued
      const uint64_t dq = sw128_desc(smem_u32(smem + C::oQ + s * C::kTile), 16, 1024);
      const uint64_t dk0 = sw128_desc(smem_u32(smem + C::oKV), 16, 1024);
      const uint64_t dv0 = sw128_desc(smem_u32(smem + C::oKV), C::kPanel, 1024);
      const uint32_t tS = tmem + s * 128, tO = tmem + C::cO + s * D;
      auto wait = [&](uint64_t *bar, uint32_t ph) {
        if (!mbar_wait(bar, ph, g)) lead = 0;
      };
      auto wait_copies = [&](const Ring<C::kStages> &r) {
        wait(&kvFull[r.st], r.ph);
        fence_proxy_async_smem();
      };
      auto give_turn = [&](int to) {
        if (lead) mbar_arrive(&bars[bPFull + to]);
      };
      auto issue_s = [&](int stage, bool pass) {
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
      wait_copies(rk);  // Q and the first K tile
      issue_s(rk.st, false);
      tc_commit_if(lead, &kvEmpty[rk.st]);
      rk.next();
      const bool pass = tiles == 2;
      for (int j = 0; j < n; ++j) {
        const Ring<C::kStages> rv = rk;  // V tile j; the next K tile follows it in the ring
        rk.next();
        wait_copies(rv);
        if (j + 1 < n) wait_copies(rk);
        const uint64_t dv = dv0 + ((rv.st * C::kTile) >> 4);
        // tile 1's turn comes from tile 0's warp at the same KV tile, tile 0's from tile 1's at the one before, or,
        // where there was none, from itself
        if (s == 0 && (j == 0 || !pass)) give_turn(0);
        wait(&bars[bPFull + s], p_ph);
        p_ph ^= 1;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_if(lead, tO, tS + kk * 8, dv + ((kk * 2048) >> 4), idO, (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit_if(lead, &kvEmpty[rv.st]);
        if (j + 1 < n) {
          issue_s(rk.st, pass);  // MMAs run in issue order: PV has read P before S overwrites it
          tc_commit_if(lead, &kvEmpty[rk.st]);
          rk.next();
        } else {
          if (pass && s == 0) give_turn(1);
          tc_commit_if(lead, &bars[bOFull + s]);
        }
      }
      // every MMA has completed before tensor memory is released (at once if none was issued)
      tc_commit_if(elect_one(), &bars[bFinal + s]);
      mbar_drain(&bars[bFinal + s], 0, g.limit_ns);
    }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int s = warp >> 2, sub = warp & 3;
    if (s < tiles) {
      const int row = row0 + s * kPackedTile + sub * 32 + lane;
      const bool real = row < rows;
      const int b = real ? row / p.group : 0, h = hk * p.group + (real ? row - b * p.group : 0);
      const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
      const uint32_t tS = tl + s * 128, tO = tl + C::cO + s * D;
      // tokens of the split that this row attends: a sequence may end inside the prefix
      const int limit =
          (real ? max(0, min(min(p.lengths[b], p.max_pages * p.page_size), p.first)) : 0) - j0 * kPackedTile;
      float m = -INFINITY;   // the maximum the row refers to (scaled, log2; -inf: nothing counted yet)
      uint64_t l2 = 0;       // its sum, in two halves
      // After an abort the loop runs on with whatever tensor memory holds: no
      // wait blocks any more, and the status word tells that O is not valid.
      for (int j = 0; j < n; ++j) {
        mbar_wait(&bars[bMask + j % kMasks], (j / kMasks) & 1, g);
        uint32_t valid[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) valid[c] = masks[(j % kMasks) * 4 + c];
        const int cols = limit - j * kPackedTile;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int k = cols - 32 * c;
          valid[c] &= k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
        }
        mbar_wait(&bars[bSFull + s], j & 1, g);
        __syncwarp();
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_nowait(tS + 32 * c, x[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_order32(x[c]);
        if (__any_sync(0xffffffffu, (valid[0] & valid[1] & valid[2] & valid[3]) != 0xffffffffu)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((valid[c] >> e) & 1u)) x[c][e] = 0xff800000u;  // -inf
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
        const bool moves = top > m + kLazy;
        if (__any_sync(0xffffffffu, moves)) {
          // the product before has completed (it did before S(j) did), so O may be rewritten here
          const float f = moves ? ex2(m - top) : 1.f;
          m = moves ? top : m;
          l2 = mul2(l2, pack2(f, f));
          if (j > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t r[16];
              tmem_ld16(tO + c0, r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st16(tO + c0, r);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), nm2 = pack2(-ref, -ref);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a0, a1;
            unpack2(fma2(pack2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sc2, nm2), a0, a1);
            a0 = ex2(a0);
            a1 = ex2(a1);
            x[c][e] = __float_as_uint(a0);
            x[c][e + 1] = __float_as_uint(a1);
            pk[e >> 1] = pack_bf16(a0, a1);
          }
          tmem_st16(tS + 16 * c, pk);
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
      float la, lb;
      unpack2(l2, la, lb);
      const float l = la + lb;
      const bool ok = mbar_wait(&bars[bOFull + s], 0, g);
      __syncwarp();
      tc_fence_after();
      // A row's result goes through this tile's place of Q, which every S has read, so that a warp's store is two
      // rows (or four) side by side and not a piece of 32; half the columns at a time, each warp its own rows.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int parts = p.parts_before + p.max_splits;
      const size_t at = ((size_t)b * p.Hq + h) * parts + split;
      constexpr int kWide = D / 2, kVecs = kWide / 4, kPer = 32 / kVecs;  // columns at a time; rows of a warp's store
      static_assert(kPackedTile * kWide * 4 == C::kTile, "a tile's rows fill its Q");
      float4 *stage = reinterpret_cast<float4 *>(smem + C::oQ + s * C::kTile) + sub * 32 * kVecs;
      const uint32_t out = __ballot_sync(0xffffffffu, real && ok);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += kWide) {
#pragma unroll
        for (int part = 0; part < kWide / 32; ++part) {
          uint32_t r[32];
          tmem_ld32(tO + c0 + 32 * part, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t *v = r + 4 * e;
            stage[lane * kVecs + ((8 * part + e) ^ (lane & (kVecs - 1)))] =
                make_float4(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv, __uint_as_float(v[2]) * inv,
                            __uint_as_float(v[3]) * inv);
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 32 / kPer; ++i) {
          const int from = kPer * i + lane / kVecs, c = lane % kVecs;
          const size_t to = __shfl_sync(0xffffffffu, (unsigned long long)at, from);
          if ((out >> from) & 1u)
            *reinterpret_cast<float4 *>(p.part_o + to * D + c0 + 4 * c) = stage[from * kVecs + (c ^ (from & (kVecs - 1)))];
        }
        __syncwarp();
      }
      if (real && ok) p.part_ml[at] = make_float2(m, l);
      tc_fence_before();
    }
  }
  __syncwarp();
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
  cudaError_t e = cudaFuncGetAttributes(&fa, dash_prefix_kernel<D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split counts on it
  return cudaFuncSetAttribute(dash_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
}

}  // namespace

cudaError_t prepare_shared() {
  const cudaError_t e = prepare_t<64>();
  return e != cudaSuccess ? e : prepare_t<128>();
}

cudaError_t launch_decode_shared(int D, const SharedParams &p, int num_sms, cudaStream_t stream) {
  const dim3 grid(p.parts_before, (unsigned)(((long long)p.B * p.group + 2 * kPackedTile - 1) / (2 * kPackedTile)),
                  p.Hkv);
  const cudaError_t e =
      D == 64 ? launch(dash_prefix_kernel<64>, grid, kThreads, smem_bytes<64>(), stream, nullptr, p)
              : launch(dash_prefix_kernel<128>, grid, kThreads, smem_bytes<128>(), stream, nullptr, p);
  return e != cudaSuccess ? e : launch_decode(D, p, num_sms, stream);
}

}  // namespace dash
