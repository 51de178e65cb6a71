// Decode attention over the 8-bit paged cache for calls that fill the GPU: the
// products on the 5th-generation tensor cores, with the codes as they lie.
//
// Per sequence, K/V head and split, over tiles of 128 tokens (scales a_t of K,
// c_t of V, up to 8 Q heads of the group):
//   x_t = scale log2(e) a_t (q . k_t),  l += 2^(x_t - m),  O += 2^(x_t - M) c_t v_t,
// m and M the running maxima of x_t and x_t + log2 c_t.  The codes are the large
// operand and need no widening; what meets them, Q and the weights, is split
// into two e4m3 terms of 4 bits each, the second 16 times larger:
//   y = y1 + y2 / 16,  y1 = e4m3(y), y2 = e4m3(16 (y - y1)),
// which are columns of their own, so that their scales stay apart until the sums
// are 32-bit:
//   S^T [128 tokens x 16] = K [128 x D] Q^T,  O^T [D x 16] += V^T [D x 128] P^T,
// columns (term, head).  Two terms hold Q's 8 bits: exactly down to 2^-13 of its
// row's largest value, and to 2^-21 of that below (the largest lands at 2^7 to
// 2^8, and a term's last place is 2^-9).  A weight is off by at most 2^-8 of
// itself, as one rounded to bf16 would be, or, where that is more, by 2^-18 of the
// one that M was set by (M goes by x_t + log2 c_t, so that it is what counts in O,
// whatever the scales of V are).  So that this does not add up over a long split,
// behind a token that outweighs all that follow it, M is set anew, down as well as
// up, at every 8th tile: 1024 tokens together lose 2^-8 of that one weight at most.
// (With an M that only rises, splits of 4096 tokens lost up to 1.6 % and splits of
// 16384 up to 6 %.)  O is a 32-bit sum: it takes an M of up to 2^64 below the largest
// one, but what stands 2^-24 and more under O itself the tensor cores cut off, as in
// any such sum; of a million tokens, in splits of 16384, that is 2^-10 at most.  l
// sums the unrounded 2^(x_t - m), and m only rises.
//
// The bound is HBM: 2 (D + 4) bytes a token and K/V head.  On the plain pipes the
// widening alone takes half the issue slots (cache8.cu's kernel stays at 60 % of
// the copy rate); here a token costs a softmax thread's instructions for its 8
// heads, once.  66 sequences of 460000 tokens, 8 K/V heads of 128: 163 us, 5.8
// TB/s or 86 % of the copy rate (rows fetched by 16-byte copies alone: 182); 32
// of 8192: 94 us (87 %); 64 of 4096 with D = 64: 81 us (52 %).  With three
// quarters of the softmax's work left out these take 160, 92 and 69: what is left
// is, at D = 128, an item's start and end, at D = 64 also a tile's chain from
// scores to weights, which half as many bytes do not shorten.
//
// A persistent CTA, two on an SM, walks its items (longest splits first) without
// a break in its loads.  Warps: 0-3 softmax (a thread owns a token, and in the
// end a dim), 4-7 fetch and split Q, 8 issues the MMAs, the next tile's scores
// before this tile's O.  A token's row lies wherever its page does.  Where a tile's
// tokens all count, TMA takes the tokens of a page at once (pages of a multiple of 8
// tokens); other rows come by 16-byte asynchronous copies, which can
// leave zeros for a token that does not count.  Tensor memory: S twice at 0 and 16, O at 32.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache8.h"
#include "decode.cuh"
#include "drain.h"
#include "fp8.cuh"
#include "sm103.cuh"

namespace dash {

using namespace dev;

namespace {

constexpr int kThreads = 384;
constexpr int kFetch = 4;  // warps that fetch, 32 rows each
constexpr int kMma = 8;    // the warp that issues; 9-11 make the warpgroup whole
constexpr int kRegsLaunch = 80, kRegsSoftmax = 128, kRegsFetch = 80, kRegsMma = 32;
static_assert(kRegsSoftmax + kRegsFetch + kRegsMma <= 3 * kRegsLaunch, "register split exceeds the CTA's allocation");
// the fetching warps keep what they were launched with: they execute no setmaxnreg
static_assert(kRegsFetch == kRegsLaunch && kRegsMma < kRegsLaunch && kRegsSoftmax > kRegsLaunch, "inc and dec as they are used");
constexpr int kHeads = 8, kTerms = 2, kCols = kTerms * kHeads;
constexpr int kTile8 = 128;        // tokens
constexpr int kSlots = 8;          // tiles whose scales and masks are held
// log2 of where a head's largest weight is put, of how far a weight may grow past
// that (e4m3 holds 448), and of how far 2^(x - m) may.
constexpr float kTopLog = 4.f, kGrow = 4.f, kLazy = 8.f;
// Tiles after which M is set anew (as many as splits of sequences of up to 65536 tokens have: no step more for those;
// looking for low tiles at each one: 66 sequences 3 % slower, 64 of 4096 at D = 64 11 %), and how far M may fall.
constexpr int kAgain = 8;
constexpr float kMostDrop = 64.f;

constexpr uint32_t kRing = 5 * 128 * kTile8;    // bytes of K and V tiles
constexpr uint32_t kColBytes = kCols * 128;     // Q or P: a row of 128 bytes for each column
constexpr uint32_t oKV = 0;
constexpr uint32_t oQ = oKV + kRing;                   // twice
constexpr uint32_t oP = oQ + 2 * kColBytes;            // twice
constexpr uint32_t oScale = oP + 2 * kColBytes;        // [kSlots][2][128]
constexpr uint32_t oMask = oScale + kSlots * 2 * kTile8 * 4;  // [kSlots][4]
constexpr uint32_t oSc = oMask + kSlots * 16;          // [2][8] a score's factor
constexpr uint32_t oItem = oSc + 2 * kHeads * 4;       // [2] what the item is
constexpr uint32_t oRed = oItem + 2 * 32;              // [16][4] maxima of the warps, then masks of heads [4]
constexpr uint32_t oSum = oRed + 4 * 16 * 4 + 16;      // [8][4] sums of the warps
constexpr uint32_t oHead = oSum + 4 * kHeads * 4;      // [8] the state of each head
constexpr uint32_t oMove = oHead + 32 * kHeads;        // [8] {l's, O's} factors of a step that moves maxima; in the end O's
constexpr uint32_t oBar = oMove + 8 * kHeads;
enum {
  bSFull = 0, bPFull = 2, bPvDone = 4, bQFull = 6, bQEmpty = 8, bTile = 10, bKvFull = bTile + kSlots,
  bKvEmpty = bKvFull + 10, bFinal = bKvEmpty + 10, kBars  // up to 10 stages
};
// K and V tiles: rows of D bytes, swizzled within 128 bytes or within 64.
template <int D>
struct Tile {
  static constexpr uint32_t kBytes = kTile8 * D, kGroup = 8 * D;  // a stage; eight rows, the unit of the layout
  static constexpr int kStages = kRing / kBytes;
  static_assert(kStages <= 10, "barriers");
  // K of tile j + n is asked for once the load kStages before it has been read.  V of tile j is read after the tile's
  // scales are, and 2 n - 3 loads lie between the two, so n reaches (kStages + 2) / 2.
  static_assert(kSlots > (kStages + 2) / 2, "a slot would be filled before it is read");
  // The fetching warps take tiles in turn, kPer of them together (all four: 3 % slower, 9 % at D = 64; each by itself,
  // with the ten stages of D = 64: 20 % slower).  A warp that waits for a stage goes by the parity of
  // its phase, so it has to know already that the phase before that has ended: its last load was at most
  // 2 kUnits - 1 loads ago, and waited for the one kStages before it.
  static constexpr int kPer = 2, kUnits = kFetch / kPer, kGroups = 4 / kPer;
  static_assert(2 * kUnits - 1 <= kStages, "a phase could be taken for the one two before it");
  // where 16-byte piece c of a row stands in it
  static __device__ __forceinline__ int place(int row, int c) { return (c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4; }
  // Descriptors.  K's rows are the operand's rows.  V's are its columns: of D = 64
  // the upper half of the 128 rows that an MMA has is the lower half again (an
  // offset of 0 between the panels of 64), and nobody reads what comes of it.
  static __device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t panel) {
    const uint64_t d = sw128_desc(addr, panel, kGroup);
    return D == 128 ? d : (d & ~(7ull << 61)) | 4ull << 61;  // 64-byte swizzle
  }
};
constexpr uint32_t oMisc = oBar + kBars * 8;
constexpr int kSorted = 256;  // sequences whose lengths are held and sorted (1024: 1000 of up to 600 tokens 90 us instead of 70)
constexpr uint32_t oLast = oMisc + 16;  // [10] the last load of each stage
constexpr uint32_t oLens = oLast + 48;
constexpr uint32_t kSmem = oLens + 4 * kSorted;
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs on an SM");
constexpr uint32_t cS = 0, cO = 2 * kCols, kTmem = 64;

// D[tmem] (+)= A[smem] * B[smem], 8-bit operands
__device__ __forceinline__ void mma8_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// Instruction descriptor: e4m3 operands, 32-bit sums; a_mn: A is MN-major.
__host__ __device__ constexpr uint32_t idesc8(int M, int N, int a_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Whether any of the 128 softmax threads says so.
__device__ __forceinline__ bool any_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// Two columns of the warp's 32 lanes, waited on.
__device__ __forceinline__ float2 tmem_ld1x2(uint32_t a, uint32_t b) {
  float2 r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%2];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%3];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b)
      : "memory");
  return r;
}
// A head of the item in hand, the same for all 128 tokens of a tile.
struct Head {
  float factor;          // of its scores
  float ref, limit;      // what 2^(x - m) refers to (m, or 0), and from where m moves
  float wref, wlimit;    // the same of the weights: M less kTopLog, or 0
  float m, M, top;       // top: the largest M so far
};
static_assert(sizeof(Head) == 32, "two 16-byte words");
// Reduces N values (a power of two up to 32) over the lanes of a warp, all at
// once: each exchange halves the values that a lane keeps.  The lane ends with
// value number lane / (32 / N); lanes of the same number hold the same.
template <int N, class Op>
__device__ __forceinline__ float reduce_all(float (&v)[N], int lane, Op op) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool high = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = high ? v[i] : v[n + i], keep = high ? v[n + i] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  for (; o > 0; o /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

// The terms of two values, as codes: term k in bytes {a, b} of t[k].
__device__ __forceinline__ void terms_of(float a, float b, uint32_t (&t)[kTerms]) {
#pragma unroll
  for (int k = 0; k < kTerms; ++k) {
    t[k] = narrow8(a, b);
    if (k + 1 < kTerms) {
      const uint32_t w = widen8(t[k]);
      const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
      a = (a - v.x) * 16.f;
      b = (b - v.y) * 16.f;
    }
  }
}

// Items of a CTA: (split, K/V head) numbers item, item + grid, ..., numbered by
// their size, so that what a CTA is dealt last is small: splits of more than
// kind / 2 and up to `kind` tokens, sequence by sequence, for each power of two
// down to a tile (of up to kSorted sequences; of more, all in one walk).  A warp
// scans 32 sequences at a time and remembers how far it got.
struct Walk {
  long long base = 0;  // splits before the block of sequences b0
  int b0 = 0, kind, at = -1;
  int n = 0, upto = 0, total = 0, whole = 0, full = 0;  // of the lane's sequence: splits of the kind, those up to it, of
                                                        // the block; whole splits of the kind, and of any
  int len_of = 0;      // the lane's sequence's tokens
  const int *lens;     // up to kSorted sequences' tokens in shared memory
  int b, split, len;   // found: the sequence, its split, its tokens

  __device__ __forceinline__ Walk(const DecodeParams &p, const int *lens)
      : kind(p.B <= kSorted ? decode_chunk(p.max_pages * p.page_size, p.least_chunk) : 0), lens(lens) {
    while (kind > kTile8 && kind / 2 >= p.max_pages * p.page_size) kind /= 2;  // there is none as long
  }
  // All lanes of a warp ask together.
  __device__ __forceinline__ bool find(const DecodeParams &p, long long want, int lane) {
    while (true) {
      if (at != b0) {
        const int mine = b0 + lane;
        n = whole = full = 0;
        if (mine < p.B) {
          len_of = kind == 0 ? decode_len(p, mine) : lens[mine];
          const int chunk = decode_chunk(len_of, p.least_chunk);
          full = len_of >> (31 - __clz(chunk));
          const int rest = len_of & (chunk - 1);
          whole = kind == 0 || kind == chunk ? full : 0;
          // the rest, or the one item of an empty sequence
          n = whole + ((rest > 0 || len_of == 0) && (kind == 0 || (rest <= kind && (rest > kind / 2 || kind <= kTile8))));
        }
        upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
        at = b0;
      }
      if (want < base + total) {
        const int off = (int)(want - base);
        const int src = __popc(__ballot_sync(0xffffffffu, upto <= off));
        b = b0 + src;
        const int i = off - __shfl_sync(0xffffffffu, upto - n, src);
        split = i < __shfl_sync(0xffffffffu, whole, src) ? i : __shfl_sync(0xffffffffu, full, src);
        len = __shfl_sync(0xffffffffu, len_of, src);
        return true;
      }
      base += total;
      b0 += 32;
      at = -1;
      if (b0 >= p.B) {
        b0 = 0;
        if (kind <= kTile8) return false;  // nothing shorter, or all in one walk
        kind >>= 1;
      }
    }
  }
};

// An item, as the fetching warps tell it to the others with its Q.
struct Item {
  int b, hk, split, n_splits, begin, end;
  int tiles;  // -1: there is none behind the last
  int pad;
};
static_assert(sizeof(Item) == 32, "a place in shared memory");
__device__ __forceinline__ Item item_of(const DecodeParams &p, const Walk &w, int head) {
  Item it;
  it.b = w.b, it.hk = head, it.split = w.split;
  const int chunk = decode_chunk(w.len, p.least_chunk);
  it.n_splits = max(1, decode_splits(w.len, p.least_chunk));
  it.begin = it.split * chunk;
  it.end = min(w.len, it.begin + chunk);
  it.tiles = (it.end - it.begin + kTile8 - 1) / kTile8;  // 0: an empty sequence
  it.pad = 0;
  return it;
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
__global__ void __launch_bounds__(kThreads, 2) dash_decode8_wide_kernel(
    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Decode8Params p,
    int box) {  // tokens that TMA takes at once; 0: none
  using Ti = Tile<D>;
  constexpr int kStages = Ti::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the join may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = warp_id(), lane = threadIdx.x & 31;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + oBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + oMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + oMisc + 4);
  float *scales = reinterpret_cast<float *>(smem + oScale);
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + oMask);
  float *factors = reinterpret_cast<float *>(smem + oSc);
  Item *items = reinterpret_cast<Item *>(smem + oItem);
  volatile int *last = reinterpret_cast<volatile int *>(smem + oLast);
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemMisaligned);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[bSFull + s], 1);
      mbar_init(&bars[bPFull + s], 1);
      mbar_init(&bars[bPvDone + s], 1);
      mbar_init(&bars[bQFull + s], kFetch);
      mbar_init(&bars[bQEmpty + s], 5);  // the MMA warp and the softmax warps
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(&bars[bTile + s], 33 * Ti::kPer);  // the copies' ends and the masks
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[bKvFull + s], 32 * Ti::kPer);
      mbar_init(&bars[bKvEmpty + s], 1);
    }
    mbar_init(&bars[bFinal], 1);
    for (int s = 0; s < kStages; ++s) last[s] = -1;
    *abort_flag = 0;
    fence_mbar_init();
  }
  int *lens = reinterpret_cast<int *>(smem + oLens);
  if (p.B <= kSorted)
    for (int b = threadIdx.x; b < p.B; b += kThreads) lens[b] = decode_len(p, b);
  if (warp == kMma) {
    tmem_alloc(tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, p.status, (uint64_t)p.spin_limit_ns};
  int ib = 0;            // the item's place, and its Q's
  uint32_t iph = 0;      // and its phase
  uint32_t T = 0;        // tiles before this item

  if (warp >= 4 && warp < kMma) {
    // ------------------------------------------------------ loads, and Q
    const int w = warp - 4, row = w * 32 + lane;
    constexpr int kPer = Ti::kPer, kUnits = Ti::kUnits, kGroups = Ti::kGroups;
    const int mine = (w % kPer) * 32 * kGroups + lane;  // the lane's first token of a tile that its warp takes part in
    constexpr int kChunks = D / 16, kRowsPer = 32 / kChunks;  // 16-byte pieces of a row, rows of a warp's copy
    const int c = lane % kChunks, rsub = lane / kChunks;
    constexpr int kLanes = D / 8;  // of a head of Q
    const int head = row / kLanes, dim = lane % kLanes * 8;
    Walk walk(p, lens);
    // split and head of the next item, and the steps to the one after it
    long long want = blockIdx.x / p.Hkv;
    int hk = blockIdx.x % p.Hkv;
    const int want_step = gridDim.x / p.Hkv, hk_step = gridDim.x % p.Hkv;
    // The next item that has tokens, with what its start waits for: its Q and the pages of the warp's first tile.
    // Empty sequences are answered on the way.
    struct Next {
      Item it;
      uint4 q;
      int page[kGroups];
    } next;
    // A lane holds the pages of the warp's tokens lane, lane + 32, ... of a tile.
    auto pages_of = [&](const Item &it, int j, int (&page)[kGroups]) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int t = it.begin + j * kTile8 + mine + 32 * i;
        page[i] = t < it.end ? p.table[it.b * p.table_row + quotient(p.page, t)] : -1;
      }
    };
    // the warp's first tile of an item with `before` tiles before it
    auto first_of = [&](uint32_t before) { return (int)((w / kPer - before) & (kUnits - 1)); };
    auto look_up = [&](uint32_t before) {
      while (true) {
        next.it.tiles = -1;
        if (!walk.find(p, want, lane)) return;
        next.it = item_of(p, walk, hk);
        want += want_step;
        hk += hk_step;
        if (hk >= p.Hkv) {
          hk -= p.Hkv;
          ++want;
        }
        if (next.it.tiles > 0) break;
        for (int h = 0; h < p.group; ++h) {
          const int hh = next.it.hk * p.group + h;
          if (row < D) p.o[next.it.b * p.o_batch + hh * p.o_head + row] = __float2bfloat16_rn(0.f);
          if (row == 0 && p.lse) p.lse[(size_t)next.it.b * p.Hq + hh] = -INFINITY;
        }
      }
      next.q = make_uint4(0u, 0u, 0u, 0u);
      if (head < p.group)
        next.q = *reinterpret_cast<const uint4 *>(p.q + next.it.b * p.q_batch +
                                                  (long long)(next.it.hk * p.group + head) * p.q_head + dim);
      pages_of(next.it, first_of(before), next.page);
    };
    look_up(0);
    while (true) {
      const Item it = next.it;
      // Q's largest value is put at 2^7 to 2^8; a head with a NaN or an infinity is all NaN
      mbar_wait(&bars[bQEmpty + ib], iph ^ 1, g);
      __syncwarp();
      if (it.tiles > 0) {
        const uint32_t x[4] = {next.q.x, next.q.y, next.q.z, next.q.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int f = min(253, 261 - (int)(top >> 7));
        const float up = top < 0x7f80u ? pow2_field(f) : NAN;
        uint32_t codes[kTerms][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t t2[kTerms];
          terms_of(__uint_as_float(x[i] << 16) * up, __uint_as_float(x[i] & 0xffff0000u) * up, t2);
#pragma unroll
          for (int n = 0; n < kTerms; ++n) codes[n][i >> 1] = i & 1 ? codes[n][i >> 1] | t2[n] << 16 : t2[n];
        }
        if (head < kHeads) {
#pragma unroll
          for (int i = 0; i < kTerms; ++i) {
            const int n = i * kHeads + head;
            *reinterpret_cast<uint2 *>(smem + oQ + ib * kColBytes + n * 128 + (((dim >> 4) ^ (n & 7)) << 4) +
                                       (dim & 15)) = make_uint2(codes[i][0], codes[i][1]);
          }
          if (dim == 0) factors[ib * kHeads + head] = p.scale_log2 * pow2_field(254 - f);
        }
        fence_proxy_async_smem();
      }
      if (row == 0) items[ib] = it;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bQFull + ib]);
      if (it.tiles < 0) break;
      const uint8_t *kbase = p.c.k + it.hk * p.c.ks.head + 16 * c, *vbase = p.c.v + it.hk * p.c.vs.head + 16 * c;
      const float *ksbase = p.c.k_scale + it.hk * p.c.kss.head, *vsbase = p.c.v_scale + it.hk * p.c.vss.head;
      // The rows of the item's tile j of K (with the scales of both) or V: load number `pos` of the CTA.
      auto fetch = [&](bool is_v, uint32_t pos, int j, const int (&page)[kGroups]) {
        const int st_at = pos % kStages;
        mbar_wait(&bars[bKvEmpty + st_at], (pos / kStages & 1) ^ 1, g);
        // After an abort nothing more arrives at a stage: one that waits for bytes of TMA has no arrivals left to take.
        if (warp_aborted(g)) return;
        if (lane == 0) last[st_at] = (int)pos;
        const CacheStrides &st = is_v ? p.c.vs : p.c.ks;
        uint8_t *const stage = smem + oKV + st_at * Ti::kBytes;
        uint64_t *bar = &bars[bKvFull + st_at];
        const int t0 = it.begin + j * kTile8;
        uint32_t valid[kGroups];
        int off[kGroups];
        bool all = true;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const int t = t0 + mine + 32 * i;
          const bool ok = page[i] >= 0 && page[i] < p.n_pages;
          if (!is_v && t < it.end && !ok) atomicCAS(p.status, 0, kStatusBadPage);
          off[i] = t - quotient(p.page, t) * p.page_size;
          valid[i] = __ballot_sync(0xffffffffu, ok);
          all = all && valid[i] == 0xffffffffu;
        }
        // TMA: where all of the warp's tokens count, and with it, as a box may reach into another warp's, all of the tile's
        const bool by_copies = !(box > 0 && all && (box <= 32 * kGroups || t0 + kTile8 <= it.end));
        if (!by_copies) {
          int n = 0;
#pragma unroll
          for (int i = 0; i < kGroups; ++i) n += ((mine + 32 * i) & (box - 1)) == 0;
          if (n > 0) mbar_arrive_expect_tx(bar, n * box * D);
          else mbar_arrive(bar);
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            if (((mine + 32 * i) & (box - 1)) == 0)
              tma_load_4d(stage + (mine + 32 * i) * D, is_v ? &tmV : &tmK, bar, 0, it.hk, off[i], page[i]);
        } else {
          const uint8_t *base = is_v ? vbase : kbase;
#pragma unroll 1
          for (int i = 0; i < kGroups; ++i) {
            int pg_i = page[0], off_i = off[0];
            uint32_t valid_i = valid[0];
#pragma unroll
            for (int k = 1; k < kGroups; ++k)
              if (i == k) pg_i = page[k], off_i = off[k], valid_i = valid[k];
            const uint32_t dst = smem_u32(stage) + (mine - lane + 32 * i + rsub) * D;
            if (valid_i == 0xffffffffu && p.whole) {
              const long long step = kRowsPer * st.token;
#pragma unroll
              for (int half = 0; half < 2; ++half) {  // 16 tokens lie in one page
                const int pg = __shfl_sync(0xffffffffu, pg_i, 16 * half), of = __shfl_sync(0xffffffffu, off_i, 16 * half);
                const uint8_t *from = wide_add(wide_add(base, pg, (int)st.page), of + rsub, (int)st.token);
#pragma unroll
                for (int k = 0; k < 16 / kRowsPer; ++k, from += step) {
                  const int rr = 16 * half + k * kRowsPer;
                  cp_async<16>(dst + rr * D + Ti::place(rr + rsub, c), from);
                }
              }
            } else {
              const long long a = (valid_i >> lane) & 1u ? pg_i * st.page + off_i * st.token : 0;
#pragma unroll
              for (int k = 0; k < 32 / kRowsPer; ++k) {
                const int rr = k * kRowsPer + rsub;
                const long long x = __shfl_sync(0xffffffffu, a, rr);
                cp_async_if<16>(dst + k * kRowsPer * D + Ti::place(rr, c), base + x, (valid_i >> rr) & 1u);
              }
            }
          }
        }
        if (!is_v) {
          const uint32_t slot = (T + j) % kSlots;
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            const bool ok = (valid[i] >> lane) & 1u;
            const uint32_t sd = smem_u32(scales + slot * 2 * kTile8 + mine + 32 * i);
            cp_async_if<4>(sd, ok ? ksbase + page[i] * p.c.kss.page + off[i] * p.c.kss.token : ksbase, ok);
            cp_async_if<4>(sd + kTile8 * 4, ok ? vsbase + page[i] * p.c.vss.page + off[i] * p.c.vss.token : vsbase, ok);
          }
          // the slot's last tile has been read (see kSlots)
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) masks[slot * 4 + (w % kPer) * kGroups + i] = valid[i];
            mbar_arrive(&bars[bTile + slot]);
          }
          cp_arrive(&bars[bTile + slot]);
        }
        if (by_copies) cp_arrive(bar);
      };
      // In the order of loads V of a tile follows K of the next one.
      int page[kGroups], after[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) page[i] = next.page[i];
      int j = first_of(T);
      bool ahead = false;
      do {
        if (j < it.tiles) fetch(false, 2 * T + (j > 0 ? 2 * j - 1 : 0), j, page);
        pages_of(it, j + kUnits, after);
        if (!ahead) look_up(T + it.tiles);
        ahead = true;
        if (j < it.tiles) fetch(true, 2 * T + (j + 1 < it.tiles ? 2 * j + 2 : 2 * j + 1), j, page);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) page[i] = after[i];
        j += kUnits;
      } while (j < it.tiles);
      T += it.tiles;
      ib ^= 1;
      if (ib == 0) iph ^= 1;
    }
    cp_wait_all();
    // what TMA still has in flight lands before the CTA exits
    named_bar(3, 32 * kFetch);  // nothing more is issued
    // (after an abort a stage at which a warp has not arrived never completes)
    drain_all(
        kStages, [&](int s) { return last[s] < 0 || mbar_test(&bars[bKvFull + s], last[s] / kStages & 1); },
        [] { return globaltimer_ns(); }, g.limit_ns);
  } else if (warp >= kMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kMma) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t idS = idesc8(128, kCols, 0), idO = idesc8(128, kCols, 1);
    Ring<kStages> r;
    uint32_t lead = elect_one();  // 0 in every lane once a wait has failed: nothing more is issued
    const uint64_t k0 = Ti::desc(smem_u32(smem + oKV), 16), v0 = Ti::desc(smem_u32(smem + oKV), 0);
    const uint64_t q0 = sw128_desc(smem_u32(smem + oQ), 16, 1024), p0 = sw128_desc(smem_u32(smem + oP), 16, 1024);
    auto wait = [&](uint64_t *bar, uint32_t ph) {
      if (!mbar_wait(bar, ph, g)) lead = 0;
    };
    while (true) {
      wait(&bars[bQFull + ib], iph);
      const int tiles = items[ib].tiles;
      if (tiles < 0 || warp_aborted(g)) break;
      __syncwarp();
      auto issue_s = [&](uint32_t tile) {
        wait(&bars[bKvFull + r.st], r.ph);
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t a = k0 + ((r.st * Ti::kBytes) >> 4), b = q0 + ((ib * kColBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) mma8_if(lead, tmem + cS + (tile & 1) * kCols, a + 2 * kk, b + 2 * kk, idS, kk > 0);
        tc_commit_if(lead, &bars[bSFull + (tile & 1)]);
        tc_commit_if(lead, &bars[bKvEmpty + r.st]);
        r.next();
      };
      issue_s(T);
      if (tiles == 1) tc_commit_if(lead, &bars[bQEmpty + ib]);
      for (int j = 0; j < tiles; ++j) {
        const uint32_t tile = T + j;
        // its place of S was read before the weights of the tile before this one came
        if (j + 1 < tiles) {
          issue_s(tile + 1);
          if (j + 2 == tiles) tc_commit_if(lead, &bars[bQEmpty + ib]);
        }
        wait(&bars[bKvFull + r.st], r.ph);
        fence_proxy_async_smem();
        wait(&bars[bPFull + (tile & 1)], (tile >> 1) & 1);
        tc_fence_after();
        const uint64_t a = v0 + ((r.st * Ti::kBytes) >> 4), b = p0 + (((tile & 1) * kColBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile8 / 32; ++kk)
          mma8_if(lead, tmem + cO, a + kk * (4 * Ti::kGroup >> 4), b + 2 * kk, idO, (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit_if(lead, &bars[bPvDone + (tile & 1)]);
        tc_commit_if(lead, &bars[bKvEmpty + r.st]);
        r.next();
      }
      T += tiles;
      ib ^= 1;
      if (ib == 0) iph ^= 1;
    }
    // every MMA has completed before tensor memory is released (at once if none was issued)
    tc_commit_if(elect_one(), &bars[bFinal]);
    mbar_drain(&bars[bFinal], 0, g.limit_ns);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int tok = threadIdx.x;
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    float *red = reinterpret_cast<float *>(smem + oRed), *sums = reinterpret_cast<float *>(smem + oSum);
    Head *heads = reinterpret_cast<Head *>(smem + oHead);
    float2 *moves = reinterpret_cast<float2 *>(smem + oMove);
    while (true) {
      mbar_wait(&bars[bQFull + ib], iph, g);
      const Item it = items[ib];
      if (tok < kHeads)
        heads[tok] = {factors[ib * kHeads + tok], 0.f, -INFINITY, 0.f, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (any_of_128(it.tiles < 0 || *g.abort)) break;  // one answer, as barriers follow
      if (lane == 0) mbar_arrive(&bars[bQEmpty + ib]);
      float l[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) l[h] = 0.f;
      // After an abort the loop runs on with whatever tensor memory holds: no
      // wait blocks any more, and the status word tells that O is not valid.
      for (int j = 0; j < it.tiles; ++j) {
        const uint32_t tile = T + j, slot = tile % kSlots;
        mbar_wait(&bars[bTile + slot], (tile / kSlots) & 1, g);
        const float ks = scales[slot * 2 * kTile8 + tok], lv = lg2(scales[slot * 2 * kTile8 + kTile8 + tok]);
        const bool valid = (masks[slot * 4 + warp] >> lane) & 1u;
        mbar_wait(&bars[bSFull + (tile & 1)], (tile >> 1) & 1, g);
        __syncwarp();
        tc_fence_after();
        uint32_t s[16];
        tmem_ld16(tl + cS + (tile & 1) * kCols, s);
        float x[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          const float y = fmaf(__uint_as_float(s[kHeads + h]), 1.f / 16, __uint_as_float(s[h])) * ks;
          x[h] = valid ? y * heads[h].factor : -INFINITY;
        }
        mbar_wait(&bars[bPvDone + (tile & 1)], ((tile >> 1) & 1) ^ 1, g);  // its place of P is free
        uint8_t *pt = smem + oP + (tile & 1) * kColBytes + (tok & 15);
        float pr[kHeads];
        const bool again = j > 0 && j % kAgain == 0;
        for (int turn = 0;; ++turn) {
          // the weights' terms, a byte in each column's row
          uint32_t over = 0;
#pragma unroll
          for (int h = 0; h < kHeads; h += 2) {
            float pv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 st = *reinterpret_cast<const float4 *>(&heads[h + i]);
              const float wlimit = heads[h + i].wlimit, a = x[h + i] + lv;
              over |= (x[h + i] > st.z || a > wlimit ? 1u : 0u) << (h + i);
              pr[h + i] = ex2(x[h + i] - st.y);
              pv[i] = ex2(a - st.w);
            }
            uint32_t t2[kTerms];
            terms_of(pv[0], pv[1], t2);
#pragma unroll
            for (int k = 0; k < kTerms; ++k) {
              const int n = k * kHeads + h;
              pt[n * 128 + (((tok >> 4) ^ (n & 7)) << 4)] = (uint8_t)t2[k];
              pt[(n + 1) * 128 + (((tok >> 4) ^ ((n + 1) & 7)) << 4)] = (uint8_t)(t2[k] >> 8);
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          if (turn > 0) {
            named_bar(2, 128);
            break;
          }
          if (!any_of_128(over != 0 || again)) break;
          // Maxima move, of the heads that need it only, so that a head's bits do not depend on the others; then the
          // weights are made anew.
          float both[2 * kHeads];
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            both[h] = x[h];
            both[kHeads + h] = x[h] + lv;
          }
          const float top = reduce_all(both, lane, [](float a, float b) { return fmaxf(a, b); });
          over = __reduce_or_sync(0xffffffffu, over);
          uint32_t *all_over = reinterpret_cast<uint32_t *>(red + 64);
          red[(lane >> 1) * 4 + warp] = top;
          if (lane == 0) all_over[warp] = over;
          named_bar(2, 128);
          if (tok < kHeads) {
            Head &hd = heads[tok];
            float2 f = make_float2(1.f, 1.f);
            if (again || ((all_over[0] | all_over[1] | all_over[2] | all_over[3]) >> tok) & 1u) {
              const float4 a = reinterpret_cast<const float4 *>(red)[tok], b = reinterpret_cast<const float4 *>(red)[kHeads + tok];
              const float m1 = fmaxf(hd.m, fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)));
              const float M1 = fmaxf(again ? hd.top - kMostDrop : hd.M, fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
              const float mr = m1 == -INFINITY ? 0.f : m1, Mr = M1 == -INFINITY ? 0.f : M1;
              f = make_float2(ex2(hd.m - mr), ex2(hd.M - Mr));
              hd.m = m1;
              hd.M = M1;
              hd.top = fmaxf(hd.top, M1);
              hd.ref = mr;
              hd.limit = m1 + kLazy;
              hd.wref = M1 == -INFINITY ? 0.f : M1 - kTopLog;
              hd.wlimit = M1 + kGrow;
            }
            moves[tok] = f;
          }
          if (j > 0) {  // the product before has completed: O may be rewritten
            mbar_wait(&bars[bPvDone + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1, g);
            __syncwarp();
            tc_fence_after();
          }
          named_bar(2, 128);
          uint32_t o[16];
          if (j > 0) tmem_ld16(tl + cO, o);
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float2 f = moves[h];
            l[h] *= f.x;
            o[h] = __float_as_uint(__uint_as_float(o[h]) * f.y);
            o[kHeads + h] = __float_as_uint(__uint_as_float(o[kHeads + h]) * f.y);
          }
          if (j > 0) {
            tmem_st16(tl + cO, o);
            tmem_st_wait();
          }
        }
        if (tok == 0) mbar_arrive(&bars[bPFull + (tile & 1)]);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) l[h] += pr[h];
      }
      // ---- the split's average, a thread a dim
      const float mine = reduce_all(l, lane, [](float a, float b) { return a + b; });
      sums[(lane >> 2) * 4 + warp] = mine;
      named_bar(2, 128);
      const int h0 = it.hk * p.group, parts = p.max_splits;
      const size_t first = ((size_t)it.b * p.Hq + h0) * parts + it.split;
      if (tok < p.group) {
        const float4 w = reinterpret_cast<const float4 *>(sums)[tok];
        const float ll = (w.x + w.y) + (w.z + w.w), m = heads[tok].m;
        // 2^(M - kTopLog - m) as a square: M may be far below m
        moves[tok] = ll == 0.f ? make_float2(0.f, 0.f)
                               : make_float2(inverse_sum(ll), ex2(0.5f * (heads[tok].M - kTopLog - m)));
        if (it.n_splits > 1) p.part_ml[first + (size_t)tok * parts] = make_float2(m, ll);
        else if (p.lse) p.lse[(size_t)it.b * p.Hq + h0 + tok] = log_sum(m, ll);
      }
      const uint32_t last = T + it.tiles - 1;
      mbar_wait(&bars[bPvDone + (last & 1)], (last >> 1) & 1, g);
      __syncwarp();
      tc_fence_after();
      named_bar(2, 128);
      float *part = p.part_o + first * D + tok;
      __nv_bfloat16 *out = p.o + it.b * p.o_batch + h0 * p.o_head + tok;
#pragma unroll 1
      for (int h = 0; h < p.group; ++h) {
        const float2 o = tmem_ld1x2(tl + cO + h, tl + cO + kHeads + h);
        const float2 f = moves[h];
        const float y = fmaf(o.y, 1.f / 16, o.x) * f.x * f.y * f.y;
        if (tok < D) {
          if (it.n_splits > 1) *part = y;
          else *out = __float2bfloat16_rn(y);
        }
        part += (size_t)parts * D;
        out += p.o_head;
      }
      tc_fence_before();
      named_bar(2, 128);  // shared memory is free for the next item
      T += it.tiles;
      ib ^= 1;
      if (ib == 0) iph ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

}  // namespace

cudaError_t prepare_decode8_wide() {
  for (auto kernel : {dash_decode8_wide_kernel<64>, dash_decode8_wide_kernel<128>}) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess && fa.numRegs != kRegsLaunch) e = cudaErrorInvalidConfiguration;  // the register split counts on it
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_decode8_wide(int D, const Decode8Params &p, int num_sms, cudaStream_t stream) {
  CUtensorMap k = {}, v = {};
  // tokens of a page that are a part of a tile
  int box = 128;
  while (p.page_size % box) box /= 2;
  if (box < 8 ||
      !encode_pages8_map(&k, p.c.k, p.n_pages, p.page_size, p.Hkv, D, p.c.ks.page, p.c.ks.token, p.c.ks.head, box) ||
      !encode_pages8_map(&v, p.c.v, p.n_pages, p.page_size, p.Hkv, D, p.c.vs.page, p.c.vs.token, p.c.vs.head, box))
    box = 0;
  return launch(D == 64 ? dash_decode8_wide_kernel<64> : dash_decode8_wide_kernel<128>, 2 * num_sms, kThreads, kSmem,
                stream, nullptr, k, v, p, box);
}

}  // namespace dash
