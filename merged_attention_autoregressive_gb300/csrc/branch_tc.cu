// fastar_branch_attention on the tensor cores (tcgen05 + TMEM, bf16).
//
// One persistent CTA per SM walks its run of units (branch.cuh; 128 keys per
// unit):
//   warps 0-7, 8-15  two softmax streams, two threads per query row: one for
//                    each half of a unit's keys, in the same TMEM lane;
//   warp 16          loader: finds the units, describes each in a ring of
//                    descriptors and fetches its key and value tiles by TMA
//                    (prefix: a 128-row box per column half; pages: a box per
//                    page and column half, one lane per page) into a ring;
//   warps 17, 18     MMA issuers: S_s = Q_s K^T (M 128, N 128, K D) and O_s +=
//                    P_s V (M 128, N D, K 128; P_s read from TMEM, where the
//                    softmax wrote it over S_s).
// Wide items (256 rows of a key/value head's queries): stream s owns rows
// 128 s .. 128 s + 127, so each tile that is fetched feeds four products, and
// one stream's softmax runs under the other's products (one issuer).  Narrow
// items (128 rows): both streams own the same rows and take the units in turn,
// each with its own O, maximum, sum and issuer (joined in TMEM at the item's
// end), which hides the softmax behind the loads of a memory-bound pass, and
// the room of the second query tile holds one more tile in flight.
//
// Both halves of a row keep one maximum, raised (and O in TMEM rescaled) only
// when a unit's exceeds it by more than 2^8, so P stays <= 256, rescaling is
// rare, and otherwise the two warps of a row only meet at a barrier.
// A unit of a branch's pages leaves the lanes of O of other branches' rows out
// of its second product: with a weight of 0 an infinity or NaN among its values
// would reach them.  Those products are slower to issue, which costs a call of
// many branches 0 to 5 % (16 tokens of 40 heads 133.6 -> 134.8 us, 64 of 5 heads a
// group 110.1 -> 110.9 us, 512 of them over 32,768 + 256 keys 407 -> 414 us, 128 of
// them 131 -> 139 us).
//
// S, maxima, sums and O are fp32; P is rounded to bf16 for the second product
// (2^-8 of each weight at most, as the inputs themselves; the sums take the
// unrounded weights).
//
// What bounds it.  Single tokens: HBM where the loads are long (16 tokens of 40
// heads over 13,460 keys: 750 MB in 135 us, 5.6 TB/s with start and join; the
// copies of a run are issued by one warp at about HBM's rate, and more of them
// in flight made some runs wait for others: 7 % slower), the chain of a stream
// where the prefix comes out of L2 (64 tokens of 5 heads a group: 1.2 us a
// unit, 111 us), start and join where they are short (4 tokens: 17.4 us).  Wide
// items: the chain of one stream - scores out of TMEM, biases, exponentials
// (2000 cycles), two products of 512 cycles each and the handovers - against
// 2048 cycles of products for both streams; 9360 queries of 12 heads over
// 41,000 keys take 1.92 to 1.97 ms by the clock under that load, 1160 TFLOP/s.  Beside the products, which read
// their operands from shared memory at its full rate, a 16-byte read of a bias
// waits 33 cycles.  Units of 64 keys with the queries in TMEM (half of that
// traffic) were slower by a quarter: the handovers then come twice as often.
//
// Waits are bounded: one that runs out sets the status word, and every warp
// leaves its loop by its own bounded waits.
#include <limits.h>
#include <math.h>

#include "branch.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kM = 128, kN = 128, kThreads = 640, kSoftmax = 16, kLoader = 16, kIssuer = 17;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // raise the running max only when exceeded by more than this (log2)

// What the consumers need of a unit: all of it in one word, but for the ends
// of items and units that some row does not see whole.
struct Desc {
  BranchUnit x;
  int bits;
};
constexpr int kAct = 3;        // streams that have rows in it
constexpr int kFull = 4;       // every row of the item sees every one of the 128 keys
constexpr int kBiased = 8;     // the keys have biases
constexpr int kFirst = 16, kLast = 32;  // of the item, in this run
constexpr int kEnd = 64;       // no unit: the run is over
constexpr int kHidden = 128;   // some of the keys' counts are 0
constexpr int kPart = 256;     // it concerns some rows of the item only: these, 9 bits each
__device__ __forceinline__ int part_of(int lo, int hi) { return kPart | lo << 9 | hi << 18; }
__device__ __forceinline__ int part_lo(int bits) { return bits >> 9 & 511; }
__device__ __forceinline__ int part_hi(int bits) { return bits >> 18 & 511; }

template <int D>
struct Shape {
  static constexpr int kTile = 128 * D * 2;              // bytes of a query, key or value tile
  static constexpr int kRing = D == 128 ? 3 : 6;         // descriptors
  static constexpr int kSlots1 = D == 128 ? 6 : 10;      // tiles in flight, one query tile
  static constexpr int kSlots2 = D == 128 ? 5 : 10;      // two query tiles
  static constexpr int kTiles = kSlots1 + 1 > kSlots2 + 2 ? kSlots1 + 1 : kSlots2 + 2;
};

template <int D>
struct Smem {
  using S = Shape<D>;
  uint8_t tiles[S::kTiles * S::kTile];  // query tiles, then the ring
  float bias[S::kRing][kN];             // log2 m of the unit's prefix rows
  Desc desc[S::kRing];
  uint64_t full[S::kSlots1], empty[S::kSlots1];
  uint64_t dfull[S::kRing], dempty[S::kRing];
  uint64_t sfull[2], pready[2], odone, qfull, fin[2];
  uint32_t tmem;
  int started1;
  uint32_t gone;                        // a bit per pair of softmax warps one of which has given up
  float row[2][kM];                     // a value per row, by stream, from one half of it to the other
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_stream(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void bar_all(int id) { asm volatile("bar.sync %0, 512;" ::"r"(id) : "memory"); }
// `threads` threads meet; whether any of them holds p.
template <int threads>
__device__ __forceinline__ bool bar_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.red.or.pred q, %1, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)p), "n"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_two(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Rows of a tile whose weight is 0 must not hold an infinity or NaN where they
// take part in a product: clears those from nk to the end of the last step of
// 16, and those of hidden keys (a bit each).  Whole warp.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* v, int nk, const uint32_t (&hidden)[4]) {
  const int lane = threadIdx.x & 31;
  auto clear = [&](int r, int c) {
    *reinterpret_cast<uint4*>(v + (c >> 3) * kN * 128 + r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
  };
  for (int e = lane; e < (-nk & 15) * (D / 8); e += 32) clear(nk + e / (D / 8), e % (D / 8));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (uint32_t w = hidden[i]; w; w &= w - 1)
      if (lane < D / 8) clear(32 * i + __ffs(w) - 1, lane);
  tc::fence_proxy_async_smem();
  __syncwarp();
}
// The hidden keys of a unit, a bit each (whole warp).
__device__ __forceinline__ void hidden_keys(const float* bias, int bits, int nk, uint32_t (&hidden)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) hidden[i] = 0u;
  if (!(bits & kHidden)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    hidden[i] = __ballot_sync(0xffffffffu, lane + 32 * i < nk && bias[lane + 32 * i] == -INFINITY);
}

// The lanes of a 128-row tile outside rows lo .. hi - 1, a bit each (whole warp).
__device__ __forceinline__ void lanes_outside(int lo, int hi, uint32_t (&off)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) off[i] = __ballot_sync(0xffffffffu, lane + 32 * i < lo || lane + 32 * i >= hi);
}
// Zeros in 32 n columns of the thread's TMEM lane (whole warp); rare, and in
// line its registers cost the softmax (16 tokens of 40 heads 136 us).
__device__ __noinline__ void clear_lanes(uint32_t taddr, int n) {
  uint32_t zero[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) zero[i] = 0u;
#pragma unroll 1
  for (int q = 0; q < n; ++q) tc::tmem_st32u(taddr + q * 32, zero);
}
// The product with the values for rows lo .. hi - 1 alone (one thread): a function
// of its own, so that the issue of the other products is as if it were not there
// (two branches of 4,680 tokens 1.93 ms, 1.97 ms with it in line).
__device__ __noinline__ void part_products(uint32_t dO, uint32_t dS, uint32_t vd, uint32_t idesc, int steps, int lo, int hi) {
  auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
  uint32_t off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) off[i] = ~below(hi - 32 * i) | below(lo - 32 * i);
#pragma unroll 2
  for (int k = 0; k < steps; ++k)
    tc::mma_bf16_tmem_a_low_rows(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc, 1u, off);
}

template <int D, bool split, bool tree>
__global__ void __launch_bounds__(kThreads, 1) branch_tc_kernel(const __grid_constant__ CUtensorMap mapPK,
                                                               const __grid_constant__ CUtensorMap mapPV,
                                                               const __grid_constant__ CUtensorMap mapK,
                                                               const __grid_constant__ CUtensorMap mapV,
                                                               const BranchArgs a, int32_t* st) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Tiles of a ring: one ring for both streams, or one each (a parity wait is
  // sound only for who has seen every earlier use of the tile, and a stream
  // that takes every other unit has not seen the other's).
  constexpr int slots = split ? S::kSlots1 / 2 : S::kSlots2;
  uint8_t* const ring = sm.tiles + (split ? 1 : 2) * S::kTile;
  // what needs nothing of the previous kernel
  branch_touch(a, st);
  if (tid == 0) {
    for (int i = 0; i < S::kSlots1; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < S::kRing; ++i) {
      tc::mbar_init(&sm.dfull[i], 1);
      tc::mbar_init(&sm.dempty[i], kSoftmax + (split ? 2 : 1));  // the softmax warps and the issuers
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.sfull[s], 1);
      tc::mbar_init(&sm.pready[s], kSoftmax / 2);
    }
    sm.gone = 0u;
    tc::mbar_init(&sm.odone, split ? 2 : 1);
    tc::mbar_init(&sm.qfull, kSoftmax);
    tc::mbar_init(&sm.fin[0], 1);
    tc::mbar_init(&sm.fin[1], 1);
    tc::fence_mbar_init();
  }
  if (warp == kIssuer + 1 && lane == 0) {
    tc::prefetch_tensormap(&mapK);
    tc::prefetch_tensormap(&mapV);
    tc::prefetch_tensormap(&mapPK);
    tc::prefetch_tensormap(&mapPV);
  }
  pdl_wait();
  const bool stopped = warp == kIssuer + 1 && status_bad(st);
  if (tid == 0 && (tc::smem_u32(sm.tiles) & 1023u)) status_set(st, FASTAR_ERR_CUDA);
  // the loader finds the run's place while the others set the CTA up
  BranchWalk w;
  bool more = false;
  if (warp == kLoader) more = w.start(a, blockIdx.x, st);
  if (warp == kIssuer) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  const int stop = __syncthreads_or(stopped || (tc::smem_u32(sm.tiles) & 1023u));
  tc::tc_fence_after();
  if (stop) {
    if (warp == kIssuer) tc::tmem_dealloc(sm.tmem, 512);
    return;
  }
  const uint32_t tmem = sm.tmem;  // S_0 / P_0, S_1 / P_1 at columns 0 and 128, O_0, O_1 at 256 and 384
  bool ok = true, bad = false;

  if (warp == kLoader) {
    // ================================================= loader
    const int box = min(1 << a.page_shift, kN);  // rows of a page box
    const int rows = a.cu[a.B] * a.g;
    uint32_t j = 0;                   // units described
    uint32_t slot0 = 0, round0 = 0;   // of the first ring: next tile, times round
    uint32_t slot1 = 0, round1 = 0;   // of the second
    uint32_t turn = 0;                // loaded units of the item
    int opened = 1;
    while (more && ok) {
      // a stretch of units of one branch, or of the prefix
      BranchUnit x;
      int count, keys_end;
      bool opens, closes;
      more = w.next(a, x, count, keys_end, opens, closes, opened);
      if (!more) break;
      opened = 0;
      if (opens) turn = 0;
      const bool own = x.branch >= 0;
      // rows of the item that it concerns, by stream
      const int r0 = x.t * a.TM;
      int lo = r0, hi = min(r0 + a.TM, rows);
      if (own) {
        lo = max(lo, x.lo * a.g);
        hi = min(hi, (x.lo + x.n) * a.g);
      }
      // keys that every row of the item sees: those of its first token, where
      // the item belongs to one branch
      int full_keys = keys_end;
      if (own)
        full_keys = x.lo * a.g <= r0 && (x.lo + x.n) * a.g >= min(r0 + a.TM, rows)
                        ? branch_limit(r0 / a.g - x.lo, x.n, x.len, a.block)
                        : 0;
      if (tree && own) full_keys = min(full_keys, x.len - x.n);
      const int part = lo < hi && (lo > r0 || hi < min(r0 + a.TM, rows)) ? part_of(lo - r0, hi - r0) : 0;
      const int acts = hi <= lo ? 0 : split ? 1 : ((lo < r0 + kM ? 1 : 0) | (hi > r0 + kM ? 2 : 0));
      // page id of box `lane` (or the counts of rows lane + 32 e) of the unit
      // at k, fetched one unit ahead
      const int32_t* table = a.table + (size_t)max(x.branch, 0) * a.max_pages;
      const int32_t* counts = a.m ? a.m + (size_t)x.h * a.C : nullptr;
      int id, cnt[4];
      auto fetch = [&](int k, int* v) {
        if (own) {
          v[0] = lane * box < kN && k + lane * box < keys_end ? table[(k + lane * box) >> a.page_shift] : -1;
        } else if (counts) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = k + lane + 32 * e;
            v[e] = p < keys_end ? counts[p] : 0;
          }
        }
      };
      int ahead[4] = {0, 0, 0, 0};
      fetch(x.k0, ahead);
      for (int i = 0; i < count && ok; ++i) {
        id = ahead[0];
#pragma unroll
        for (int e = 0; e < 4; ++e) cnt[e] = ahead[e];
        if (i + 1 < count) fetch(x.k0 + kN, ahead);
        x.nk = max(0, min(kN, keys_end - x.k0));
        const int act = x.nk > 0 ? acts : 0;
        const int ds = j % S::kRing;
        if (j >= S::kRing) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.dempty[ds], (j / S::kRing - 1) & 1u));
        if (!ok) break;
        bool hidden = false;
        if (!own && counts) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sm.bias[ds][lane + 32 * e] = cnt[e] > 0 ? __log2f((float)cnt[e]) : -INFINITY;
            hidden = hidden || (cnt[e] <= 0 && lane + 32 * e < x.nk);
          }
          hidden = __any_sync(0xffffffffu, hidden);
        }
        if (lane == 0) {
          Desc& d = sm.desc[ds];
          d.x = x;
          d.bits = act | part | (x.nk == kN && x.k0 + kN <= full_keys ? kFull : 0) | (!own && counts ? kBiased : 0) | (hidden ? kHidden : 0) |
                   (opens && i == 0 ? kFirst : 0) | (closes && i == count - 1 ? kLast : 0);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.dfull[ds]);
        ++j;
        if (act) {
          int row = x.h * a.C + x.k0;
          bool mine = lane == 0;
          uint32_t bytes = kN * D * 2;
          if (own) {
            mine = lane * box < x.nk;
            if (mine && (id < 0 || id >= a.n_pages)) {
              bad = true;
              mine = false;
            }
            row = ((id * a.H + x.h) << a.page_shift) + (x.k0 & ((1 << a.page_shift) - 1));
            bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box * D * 2;
          }
          const bool second = split && (turn++ & 1);
          uint32_t slot = second ? slot1 : slot0, round = second ? round1 : round0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t at = slot + (second ? slots : 0);
            if (round > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.empty[at], (round - 1) & 1u));
            if (!ok) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(&sm.full[at], bytes);
            __syncwarp();
            if (mine) {
              uint8_t* dst = ring + (size_t)at * S::kTile + (own ? lane * box * 128 : 0);
              const CUtensorMap* map = own ? (kv ? &mapV : &mapK) : (kv ? &mapPV : &mapPK);
#pragma unroll
              for (int c = 0; c < D / 64; ++c) tc::tma_load_2d(dst + c * kN * 128, map, &sm.full[at], c * 64, row);
            }
            if (++slot == (uint32_t)slots) {
              slot = 0;
              ++round;
            }
          }
          if (second) {
            slot1 = slot;
            round1 = round;
          } else {
            slot0 = slot;
            round0 = round;
          }
        }
        x.k0 += kN;
        if (opens && i == 0) w.record(a, false);
      }
    }
    w.record(a, true);
    // no unit: the end of the run
    if (ok) {
      const int ds = j % S::kRing;
      if (j >= S::kRing) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.dempty[ds], (j / S::kRing - 1) & 1u));
      if (ok && lane == 0) {
        sm.desc[ds].bits = kEnd;
        tc::mbar_arrive(&sm.dfull[ds]);
      }
    }
    // the copies have landed before the CTA exits, also when somebody's wait
    // ran out and nobody took the last tiles
    if (lane == 0)
      for (int i = 0; i < slots; ++i) {
        const uint32_t n0 = round0 + (i < (int)slot0), n1 = round1 + (i < (int)slot1);
        if (n0 && !tc::mbar_wait(&sm.full[i], (n0 - 1) & 1u)) ok = false;
        if (n1 && !tc::mbar_wait(&sm.full[slots + i], (n1 - 1) & 1u)) ok = false;
      }
    ok = __all_sync(0xffffffffu, ok);
  } else if (split && (warp == kIssuer || warp == kIssuer + 1)) {
    // ================================================= MMA issuers, one per stream
    // Descriptors are computed on every lane, outside the elected lane's
    // branch, and the steps are unrolled.
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kM, kN, 0, 0);
    constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kM, D, 0, 1);
    const int s = warp - kIssuer;
    const int base = s * slots;  // of the stream's ring
    const uint32_t ring_addr = tc::smem_u32(ring + (size_t)base * S::kTile);
    uint64_t *const full = sm.full + base, *const empty = sm.empty + base;
    const uint32_t qd = tc::desc_low(tc::smem_u32(sm.tiles), 16);
    const uint32_t dS = tmem + s * 128, dO = tmem + 256 + s * 128;
    uint32_t slot = 0, phase = 0;    // of the ring: the next unit's key tile
    uint32_t items = 0, turn = 0;
    uint32_t np = 0;                 // P tiles consumed
    bool pend = false;               // S is out, its P V not yet
    uint32_t pslot = 0, pphase = 0;  // its value tile
    int pk = 0;                      // its keys
    bool pclear = false;             // some value rows have to be cleared
    uint32_t phidden[4];             // its hidden keys
    int pbits = 0;                   // its descriptor's
    uint32_t acc = 0u;               // 0: O starts anew
    bool issued = false;
    auto pv = [&]() {
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[pslot], pphase) && tc::mbar_wait(&sm.pready[s], np & 1u));
      if (!ok) return;
      tc::tc_fence_after();
      const uint32_t vd = tc::desc_low(ring_addr + pslot * S::kTile, kN * 128);
      if (pclear) clear_rows<D>(ring + (size_t)(base + pslot) * S::kTile, pk, phidden);
      if (pbits & kPart) {
        // O was cleared where this is the first (see the softmax)
        const int steps = (pk + 15) / 16;
        uint32_t off[4];
        lanes_outside(part_lo(pbits), part_hi(pbits), off);
        if (tc::elect_one()) {
#pragma unroll 2
          for (int k = 0; k < steps; ++k)
            tc::mma_bf16_tmem_a_low_rows(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc_pv, 1u, off);
          tc::mma_commit(&empty[pslot]);
        }
      } else if (pk == kN) {
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < kN / 16; ++k)
            tc::mma_bf16_tmem_a_low(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc_pv, k > 0 ? 1u : acc);
          tc::mma_commit(&empty[pslot]);
        }
      } else {
        const int steps = (pk + 15) / 16;
        if (tc::elect_one()) {
          for (int k = 0; k < steps; ++k)
            tc::mma_bf16_tmem_a_low(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc_pv, k > 0 ? 1u : acc);
          tc::mma_commit(&empty[pslot]);
        }
      }
      __syncwarp();
      ++np;
      acc = 1u;
      pend = false;
    };
    for (uint32_t j = 0; ok; ++j) {
      const int ds = j % S::kRing;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.dfull[ds], (j / S::kRing) & 1u));
      if (!ok) break;
      const int bits = sm.desc[ds].bits, nk = sm.desc[ds].x.nk;
      uint32_t hidden[4];
      hidden_keys(sm.bias[ds], bits, nk, hidden);
      __syncwarp();
      if (bits & kEnd) break;
      if (lane == 0) tc::mbar_arrive(&sm.dempty[ds]);
      const int act = bits & kAct;
      if (bits & kFirst) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.qfull, items & 1u));
        if (!ok) break;
        acc = 0u;
        turn = 0;
      }
      const bool mine = act && (int)(turn & 1) == s;
      const uint32_t vslot = slot + 1 == (uint32_t)slots ? 0 : slot + 1;
      const uint32_t vphase = slot + 1 == (uint32_t)slots ? phase ^ 1u : phase;
      if (mine && pend) {
        pv();
        if (!ok) break;
      }
      if (mine) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[slot], phase));
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t kd = tc::desc_low(ring_addr + slot * S::kTile, 16);
        if (bits & kHidden) clear_rows<D>(ring + (size_t)(base + slot) * S::kTile, 0, hidden);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kN * 128 + (k & 3) * 32) / 16;
            tc::mma_bf16_low(dS, qd + off, kd + off, idesc_qk, k > 0 ? 1u : 0u);
          }
          tc::mma_commit(&sm.sfull[s]);
          tc::mma_commit(&empty[slot]);
        }
        __syncwarp();
        issued = true;
        pend = true;
        pslot = vslot;
        pphase = vphase;
        pk = nk;
        pclear = (nk & 15) || (bits & kHidden);
        pbits = bits;
#pragma unroll
        for (int i = 0; i < 4; ++i) phidden[i] = hidden[i];
      }
      if (act) ++turn;
      if (mine) {
        slot = vslot + 1 == (uint32_t)slots ? 0 : vslot + 1;
        phase = vslot + 1 == (uint32_t)slots ? vphase ^ 1u : vphase;
      }
      if (bits & kLast) {
        if (pend) pv();
        if (ok && tc::elect_one()) tc::mma_commit(&sm.odone);
        __syncwarp();
        ++items;
      }
    }
    if (issued) {
      // every product has finished before TMEM is freed
      if (tc::elect_one()) tc::mma_commit(&sm.fin[s]);
      __syncwarp();
      if (!tc::mbar_wait(&sm.fin[s], 0)) ok = false;
    }
  } else if (!split && warp == kIssuer) {
    // ================================================= MMA issuer of both streams
    // In turn P_0 V and Q_0 K^T, then P_1 V and Q_1 K^T: each softmax has the
    // other stream's two products to itself (with an issuer per stream both
    // fell into step, and the tensor core idled through both softmaxes).  The
    // queue of the tensor core holds a few MMAs only, so a stream's two
    // products go out without a wait between them: both tiles are waited for
    // first, and the next unit's descriptor is read under the queued products.
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kM, kN, 0, 0);
    constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kM, D, 0, 1);
    const uint32_t ring_addr = tc::smem_u32(ring), q_addr = tc::smem_u32(sm.tiles);
    const bool leader = tc::elect_one();
    uint32_t slot = 0, phase = 0, items = 0;
    // the streams whose S is out and whose P V is not yet, their value tile
    // (one for both), its keys, and whether O starts anew
    int pend = 0, pk = 0;
    uint32_t pslot = 0, pphase = 0, np = 0u, acc = 0u;  // np, acc: a bit per stream
    bool pclear = false;                                // some value rows have to be cleared
    int pbits = 0;                                      // its descriptor's
    bool pfast = false;                                 // all of its keys, for all rows
    uint32_t phidden[4], hidden[4];                     // hidden keys, of the tile and of the unit read
    bool issued = false;
    auto values = [&]() {
      ok = ok && tc::mbar_wait(&sm.full[pslot], pphase);
      if (pclear) clear_rows<D>(ring + (size_t)pslot * S::kTile, pk, phidden);
    };
    auto products = [&](const int s, const bool next, const bool next_last) {
      const bool old = pend >> s & 1;
      if (!old && !next) return;
      const uint32_t vd = tc::desc_low(ring_addr + pslot * S::kTile, kN * 128);
      const uint32_t kd = tc::desc_low(ring_addr + slot * S::kTile, 16);
      const uint32_t qd = tc::desc_low(q_addr + s * S::kTile, 16);
      // weights: keys 0-63 over S columns 0-31, keys 64-127 over columns 64-95
      const uint32_t dS = tmem + s * 128, dO = tmem + 256 + s * 128, ac = acc >> s & 1u;
      if (old) {
        ok = ok && tc::mbar_wait(&sm.pready[s], np >> s & 1u);
        np ^= 1u << s;
        acc |= 1u << s;
        pend &= ~(1 << s);
      }
      tc::tc_fence_after();
      if (leader && ok) {
        if (old) {
          if (pfast) {
#pragma unroll
            for (int k = 0; k < kN / 16; ++k)
              tc::mma_bf16_tmem_a_low(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc_pv,
                                      k > 0 ? 1u : ac);
          } else {
            const int steps = (pk + 15) / 16;
            if (pbits & kPart) {
              part_products(dO, dS, vd, idesc_pv, steps, part_lo(pbits) - s * kM, part_hi(pbits) - s * kM);
            } else {
              for (int k = 0; k < steps; ++k)
                tc::mma_bf16_tmem_a_low(dO, dS + (k >> 2) * 64 + (k & 3) * 8, vd + k * (16 * 128 / 16), idesc_pv,
                                        k > 0 ? 1u : ac);
            }
          }
          if (pend == 0) tc::mma_commit(&sm.empty[pslot]);  // no stream wants the tile any more
        }
        if (next) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kN * 128 + (k & 3) * 32) / 16;
            tc::mma_bf16_low(dS, qd + off, kd + off, idesc_qk, k > 0 ? 1u : 0u);
          }
          tc::mma_commit(&sm.sfull[s]);
          if (next_last) tc::mma_commit(&sm.empty[slot]);
        }
      }
      __syncwarp();
    };
    int bits = 0, nk = 0;
    bool read = false;  // the unit's descriptor has been read
    auto take = [&](uint32_t j, bool wait) {
      const int ds = j % S::kRing;
      if (wait)
        ok = ok && tc::mbar_wait(&sm.dfull[ds], (j / S::kRing) & 1u);
      else if (!__all_sync(0xffffffffu, tc::mbar_test_wait(&sm.dfull[ds], (j / S::kRing) & 1u)))
        return;
      bits = sm.desc[ds].bits;
      nk = sm.desc[ds].x.nk;
      hidden_keys(sm.bias[ds], bits, nk, hidden);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.dempty[ds]);
      read = true;
    };
    for (uint32_t j = 0;; ++j) {
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (!read) take(j, true);
      read = false;
      if (!ok || (bits & kEnd)) break;
      const int uact = bits & kAct, ubits = bits, unk = nk;
      uint32_t uhidden[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) uhidden[i] = hidden[i];
      if (ubits & kFirst) {
        ok = ok && tc::mbar_wait(&sm.qfull, items & 1u);
        acc = 0u;
      }
      if (uact) {
        if (pend) values();
        ok = ok && tc::mbar_wait(&sm.full[slot], phase);
        if (ubits & kHidden) clear_rows<D>(ring + (size_t)slot * S::kTile, 0, uhidden);
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          products(s, uact >> s & 1, (uact >> (s + 1)) == 0);
          if (s == 0) take(j + 1, false);
        }
        issued = true;
        pend = uact;
        pk = unk;
        pclear = (unk & 15) || (ubits & kHidden);
        pbits = ubits;
        pfast = unk == kN && !(ubits & kPart);
#pragma unroll
        for (int i = 0; i < 4; ++i) phidden[i] = uhidden[i];
        pslot = slot + 1 == slots ? 0 : slot + 1;
        pphase = slot + 1 == slots ? phase ^ 1u : phase;
        slot = pslot + 1 == slots ? 0 : pslot + 1;
        phase = pslot + 1 == slots ? pphase ^ 1u : pphase;
      }
      if (ubits & kLast) {
        if (pend) values();
        for (int s = 0; s < 2; ++s) products(s, false, false);
        if (leader && ok) tc::mma_commit(&sm.odone);
        __syncwarp();
        ++items;
      }
    }
    if (issued) {
      // every product has finished before TMEM is freed
      if (leader) tc::mma_commit(&sm.fin[0]);
      __syncwarp();
      if (!tc::mbar_wait(&sm.fin[0], 0)) ok = false;
    }
  } else if (warp < kSoftmax) {
    // ================================================= softmax
    const int s = warp >> 3, half = (warp >> 2) & 1;  // stream, half of the unit's keys
    const int wr = (warp & 3) * 32 + lane;            // row of the stream's tile
    const int pair = 3 + s * 4 + (warp & 3);          // barrier of the two warps of these rows
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + s * 128, tO = tl + 256 + s * 128 + half * (D / 2);
    const float scale2 = a.scale * kLog2e;
    const int rows = a.cu[a.B] * a.g;
    uint32_t ns = 0, items = 0, turn = 0;  // S tiles seen, items, active units of the item
    int r = 0;                             // the row, counted over the items of the head
    float m = -INFINITY, l = 0.f;          // of the row; of this half's keys
    bool started = false;
    // Warps meet at named barriers, which have no limit of their own.  So a
    // warp whose bounded wait ran out does not just leave: the barrier that
    // its partners come to next is always one that carries a flag, and there
    // it says so (met: how many of these meetings it has had on its way out).
    int met = 0;
    for (uint32_t j = 0; ok; ++j) {
      const int ds = j % S::kRing;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.dfull[ds], (j / S::kRing) & 1u));
      if (!ok) break;
      const int bits = sm.desc[ds].bits;
      if (bits & kEnd) break;
      const int act0 = bits & kAct;
      if (bits & kFirst) {
        const BranchUnit x = sm.desc[ds].x;
        r = x.t * a.TM + (split ? 0 : s * kM) + wr;
        // gather the row's queries (the previous item's products are done:
        // odone was waited for)
        m = -INFINITY;
        l = 0.f;
        started = false;
        turn = 0;
        const uint32_t q0 = tc::smem_u32(sm.tiles + (split ? 0 : s) * S::kTile);
        const char* src = (const char*)a.q;
        const uint32_t n = r < rows ? 16u : 0u;
        if (n) src += ((size_t)(x.h * a.g + r % a.g) * a.N + r / a.g) * (D * 2);
        // the warps of a tile's rows share its 16-byte columns
        constexpr int per = D / (split ? 32 : 16);
        const int c0 = (split ? s * 2 + half : half) * per;
#pragma unroll
        for (int c = 0; c < per; ++c)
          tc::cp_async16(q0 + tc::sw128_offset(wr, c0 + c, kM), src + (n ? (c0 + c) * 16 : 0), n);
        // the first step up the tree, for the units of drafts to come
        if (tree && r < rows) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.parent + r / a.g));
        tc::cp_async_wait_all();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.qfull);
      }
      const bool active = act0 && (split ? (turn & 1) == (uint32_t)s : (act0 >> s & 1));
      if (act0) ++turn;
      if (active) {
        int seen = 64;  // keys of this half that the row sees
        uint64_t sees = ~0ull;  // tree: which of them
        bool any = r - lane < rows, all = true, none = false;  // (warps behind the last token have nothing to do)
        if (!(bits & kFull)) {
          // rows behind the last token count as full: nobody reads their results
          seen = (r < rows ? branch_row_keys(a, sm.desc[ds].x, r) : kN) - half * 64;
          any = __any_sync(0xffffffffu, r < rows && seen + half * 64 > 0);  // alike in both halves
          if (tree) sees = r < rows ? tree_row_keys(a, sm.desc[ds].x, r, half * 64, bad) : ~0ull;
          // rows that see nothing of it beside rows that see it whole (a unit of
          // one branch among others): computed unmasked, and dropped at the end
          none = split && (tree ? sees == 0ull : seen <= 0);
          all = __all_sync(0xffffffffu, none || (tree ? sees == ~0ull : seen >= 64));
        }
        if (!started && (bits & kPart)) {
          // the product with the values leaves the other rows' O as it is, so
          // that no value of one branch reaches another's: here O begins at 0
          clear_lanes(tO, D / 64);
        }
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.sfull[s], ns & 1u));
        if (!ok) break;
        ++ns;
        tc::tc_fence_after();
        uint32_t pk[32];
        if (any) {
          // log2 scores; without a bias or a mask the raw products, whose
          // scale goes into the exponent's multiply-add
          uint32_t raw[64];
          float* const v = reinterpret_cast<float*>(raw);
          tc::tmem_ld64_async(tS + half * 64, raw);
          const bool biased = bits & kBiased;
          const bool plain = !biased && all;
          none = none && all;
          const float mul = plain ? scale2 : 1.f;
          tc::tmem_wait64(raw);
          if (!plain) {
            if (biased) {
              const float* bias = sm.bias[ds] + half * 64;
#pragma unroll
              for (int i = 0; i < 64; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(bias + i);
                tc::fma2(v[i], v[i + 1], scale2, scale2, b.x, b.y);
                tc::fma2(v[i + 2], v[i + 3], scale2, scale2, b.z, b.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 64; i += 2) tc::mul2(v[i], v[i + 1], scale2, scale2);
            }
            if (!all) {
#pragma unroll
              for (int i = 0; i < 64; ++i) v[i] = (tree ? (uint32_t)(sees >> (i & 32)) >> (i & 31) & 1u : i < seen) ? v[i] : -INFINITY;
            }
          }
          float tm[8];
#pragma unroll
          for (int i = 0; i < 64; i += 16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) tm[e] = i == 0 ? fmaxf(v[e], v[8 + e]) : tc::max3(tm[e], v[i + e], v[i + 8 + e]);
          }
          float top =
              fmaxf(tc::max3(tm[0], tm[1], tm[2]), tc::max3(tm[3], tm[4], tc::max3(tm[5], tm[6], tm[7]))) * mul;
          if (none) top = -INFINITY;
          // both halves of a row keep one maximum: while neither exceeds it by
          // more than 2^8 they only meet here
          tc::tc_fence_before();
          const bool meet = bar_or<64>(pair, top > m + kRescale);
          tc::tc_fence_after();
          if (meet) {
            if (*(volatile uint32_t*)&sm.gone >> pair & 1u) {
              ok = false;
              met = 1;
              break;
            }
            float* const shared_top = &sm.row[s][wr];
            if (half == 0) *shared_top = top;
            bar_two(pair);
            if (half == 1) *shared_top = top = fmaxf(top, *shared_top);
            bar_two(pair);
            top = *shared_top;
            const bool raise = top > m + kRescale;
            const float mn = raise ? top : m;
            const float alpha = (raise && m != -INFINITY) ? exp2f(m - mn) : 1.f;
            if (started && __any_sync(0xffffffffu, alpha != 1.f)) {
              // S of this unit was issued behind the P V of the stream's last
              // one, and products complete in issue order: O is at rest
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                float o[8];
                tc::tmem_ld8(tO + q * 8, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= alpha;
                tc::tmem_st8(tO + q * 8, o);
              }
            }
            l *= alpha;
            m = mn;
            tc::tc_fence_before();
            bar_two(pair);  // O is rescaled before either half's weights are taken
          }
          const float base = m == -INFINITY ? 0.f : -m;
          float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            tc::fma2(v[i], v[i + 1], mul, mul, base, base);
            const float p0 = ex2(v[i]), p1 = ex2(v[i + 1]);
            tc::add2(ps[i & 7], ps[(i & 7) + 1], p0, p1);
            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
            pk[i >> 1] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (!none) l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
          if (split && __any_sync(0xffffffffu, none)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = none ? 0u : pk[i];
          }
        } else {
          // no row of the warp is concerned: weights 0
#pragma unroll
          for (int i = 0; i < 32; ++i) pk[i] = 0u;
        }
        tc::tmem_st32u(tS + half * 64, pk);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.pready[s]);
        started = true;
      }
      __syncwarp();
      BranchUnit x;
      if (bits & kLast) x = sm.desc[ds].x;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.dempty[ds]);
      if (bits & kLast) {
        // ---- the item's end: O of the run
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.odone, items & 1u));
        if (!ok) break;
        if (bar_or<64>(pair, false)) {
          ok = false;
          met = 1;
          break;
        }
        ++items;
        tc::tc_fence_after();
        // the sums of both halves; O is split by columns from here on
        if (half == 0) sm.row[s][wr] = l;
        bar_two(pair);
        if (half == 1) sm.row[s][wr] = l = sm.row[s][wr] + l;
        bar_two(pair);
        l = sm.row[s][wr];
        float w0 = 1.f, w1 = 0.f;
        bool have1 = false;
        if (split) {
          // stream 1 hands its maxima and sums over; stream 0 reads both O
          float2* ml = reinterpret_cast<float2*>(sm.tiles);  // the query tile is free
          if (s == 1 && half == 0) {
            ml[wr] = make_float2(m, l);
            if (wr == 0) sm.started1 = started ? 1 : 0;
          }
          if (bar_or<512>(1, false)) {
            ok = false;
            met = 2;
            break;
          }
          if (s == 0) {
            const float2 o = ml[wr];
            have1 = sm.started1 != 0;
            const float mn = fmaxf(m, o.x), base = mn == -INFINITY ? 0.f : mn;
            w0 = m == -INFINITY && l == 0.f ? 0.f : exp2f(m - base);
            w1 = o.x == -INFINITY && o.y == 0.f ? 0.f : exp2f(o.x - base);
            l = (l == 0.f ? 0.f : l * w0) + (o.y == 0.f ? 0.f : o.y * w1);
            m = mn;
          }
        }
        if (!split || s == 0) {
          const bool whole = x.flags & 4, live = r < rows;
          const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
          w0 *= inv;
          w1 *= inv;
          const size_t at = live ? (size_t)(x.h * a.g + r % a.g) * a.N + r / a.g : 0;
          const int slot_row = (split ? 0 : s * kM) + wr;
          // a finished row goes through the place of its own queries (free by
          // now; other warps may gather the next item's already) and leaves in
          // whole lines; a partial is laid out so that the rows of a warp are
          // neighbours
          uint8_t* const stage = sm.tiles + (split ? 0 : s) * S::kTile;
          if (split && whole) bar_stream(2);  // the maxima and sums in it have been read
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            float o[32];
            if (started) {
              tc::tmem_ld32(tO + q * 32, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= w0;
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (have1) {
              float o1[32];
              tc::tmem_ld32(tO + 128 + q * 32, o1);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], w1, o[i]);
            }
            const int col = half * (D / 2) + q * 32;
            if (whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_vec<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16*>(stage + tc::sw128_offset(wr, col / 8 + i, kM)),
                                         o + i * 8);
            } else if (live) {
              float* po = a.po + (size_t)x.slot * a.slot_rows * D + ((size_t)(col / 4) * a.slot_rows + slot_row) * 4;
#pragma unroll
              for (int i = 0; i < 8; ++i) st_vec<float, 4>(po + (size_t)i * a.slot_rows * 4, o + i * 4);
            }
          }
          if (live && half == 0) {
            if (whole) {
              if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
            } else {
              a.pml[(size_t)x.slot * a.slot_rows + slot_row] = make_float2(m, l);
            }
          }
          if (whole) {
            bar_two(pair);
            constexpr int per = D / 8, step = 32 / per;  // pieces of a row, rows per warp access
            const int c = lane % per;
#pragma unroll
            for (int k = 0; k < 16; k += step) {
              const int y = half * 16 + k + lane / per;  // row of the warp's 32
              const size_t to = __shfl_sync(0xffffffffu, at, y);
              const int yr = (warp & 3) * 32 + y;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + tc::sw128_offset(yr, c, kM));
              if (r - lane + y < rows) *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + to * D + c * 8) = v;
            }
          }
        }
        if (split) {
          // stream 1 may overwrite its O (by its next P) only now
          tc::tc_fence_before();
          bar_all(11);
          tc::tc_fence_after();
        } else {
          tc::tc_fence_before();
          bar_two(pair);  // the sums and the staged rows have been read
          tc::tc_fence_after();
        }
      }
    }
    if (met == 0) {
      if (!ok && lane == 0) {
        atomicOr(&sm.gone, 1u << pair);
        __threadfence_block();
      }
      __syncwarp();
      if (bar_or<64>(pair, !ok)) ok = false;
    }
    if (split && met < 2) (void)bar_or<512>(1, !ok);
    tc::cp_async_wait_all();
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (!ok) status_set(st, FASTAR_ERR_TIMEOUT);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kIssuer) tc::tmem_dealloc(tmem, 512);
  pdl_trigger();
}

template <int D, bool split, bool tree>
int launch_t(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  CUtensorMap pk, pv, k, v;
  const uint32_t box = (1u << a.page_shift) < (uint32_t)kN ? (1u << a.page_shift) : (uint32_t)kN;
  const uint64_t rows = ((uint64_t)a.n_pages * a.H) << a.page_shift;
  // a part that is absent is never loaded; its maps describe the queries
  int rc = make_tmap_bf16_2d(&k, rows ? a.K : a.q, rows ? rows : 1, D, box, 64);
  if (rc == FASTAR_OK) rc = make_tmap_bf16_2d(&v, rows ? a.V : a.q, rows ? rows : 1, D, box, 64);
  if (rc == FASTAR_OK) rc = make_tmap_bf16_2d(&pk, a.C ? a.pK : a.q, a.C ? (uint64_t)a.H * a.C : 1, D, kN, 64);
  if (rc == FASTAR_OK) rc = make_tmap_bf16_2d(&pv, a.C ? a.pV : a.q, a.C ? (uint64_t)a.H * a.C : 1, D, kN, 64);
  if (rc != FASTAR_OK) return rc;
  constexpr int smem = (int)sizeof(Smem<D>);
  static_assert(smem <= 227 * 1024, "shared memory");
  auto kernel = branch_tc_kernel<D, split, tree>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      launch_pdl(kernel, dim3(a.G), dim3(kThreads), smem, s, pk, pv, k, v, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, tree ? "branch_tc_tree" : "branch_tc");
  return FASTAR_OK;
}

}  // namespace

template <bool tree>
static int launch_d(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  if (a.TM == kM) return a.D == 128 ? launch_t<128, true, tree>(a, st, s) : launch_t<64, true, tree>(a, st, s);
  return a.D == 128 ? launch_t<128, false, tree>(a, st, s) : launch_t<64, false, tree>(a, st, s);
}
int launch_branch_tc(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  return a.parent ? launch_d<true>(a, st, s) : launch_d<false>(a, st, s);
}

}  // namespace fastar
