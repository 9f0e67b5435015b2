// fastar_page_mass on the tensor cores (tcgen05 + TMEM, bf16).
//
// One persistent CTA per SM takes its items (page_mass.cuh), 256 keys by 128
// rows at a time.  The scores are taken transposed, S^T = K Q^T: a key is a TMEM
// lane and a row a column, so that a thread sums the weights of its key in a
// register, and nothing but 256 sums leaves an item.
// The rows' log-sum-exps enter as one more step of the product: 16 channels of the
// keys hold 1, 1, 1, 0, ... and those of a row the three bf16 parts of -lse / scale
// (24 bits), so that a column's score comes out ready for the exponential.  Read
// from shared memory instead they were 900 passes through it a unit, beside the
// 1,150 cycles that the products' operands take.
//   warps 0-15   weights: warp w takes the keys of lane quarter w % 4 of key tile
//                w / 4 % 2 and half w / 8 of the columns (eight warps a unit in turn
//                idled while their half of TMEM was filled); at an item's end the
//                second halves' sums are handed over.  Without a decay the masses
//                are added to in L2, each by one thread once;
//   warp 16      keys: a page box per lane and column half by TMA;
//   warps 17, 18 products: two of M 128, N = the live rows, K = D per unit, into
//                one of two halves of TMEM, even units by one warp and odd ones by the
//                other.  The queue of products is a few deep and a look at a barrier
//                in shared memory takes long beside them, so that one warp for all
//                left the tensor core idle for as long as it worked;
//   warps 19-22  rows: a unit each in turn.  The rows' log-sum-exps and limits are
//                read while the units before are worked on; once the query tile's
//                place is free a run of rows is fetched by TMA, others 16 bytes a
//                lane.
//
// What bounds it: the handovers between products and weights.  Two chunks of 4,680
// tokens by frames over 9,360 keys, 12 heads: 215 us, 1.04 PFLOP/s, the tensor
// pipe busy 54 % of the time and the exponentials' 50 %; without the weights' work
// the same products take 147 us, without the exponentials 186 us.  On the way there:
// query rows by 16-byte copies 448 us, by TMA 284 us; one warp for the products 255
// us; their inputs a unit less ahead 242 us; every unit through the masked loop 234
// us.  256 keys by 128 rows, because every tile of queries out of L2 then feeds two
// products; N 256 would read the keys' tile half as often, but leaves no second half
// of TMEM.
//
// Waits are bounded: one that runs out sets the status word, and every warp
// leaves its loop by its own bounded waits.
#include <math.h>

#include "page_mass.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kTK = 256, kTQ = 128, kCtas = 152;
constexpr int kWeights = 16, kKeys = 16, kProducts = 17, kRows = 19, kThreads = 23 * 32;
// A unit's log-sum-exps and limits are written after the products of the unit four
// before it, the last turn of the same warp, so after the weights of the unit six
// before it: its description has one of eight places.  Its query tile waits for the
// products of the last unit in the same place.
constexpr int kTurns = 4, kMeta = 8;
constexpr int kPlaces = 16;  // items whose page ids are kept: the keys are at most 8 items ahead of the products, and these a few units of the weights
constexpr float kLog2e = 1.4426950408889634f;

// A unit: its live rows, and whether some row does not see every key, or is nobody's.
constexpr int kMasked = 256;

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;                        // bytes of 128 keys or rows
  static constexpr int kQ = D == 128 ? 3 : 4;                      // query tiles (two of 128 channels: 224 us, three: 215 us)
  static constexpr int kSlots = (D == 128 ? 6 : 12) - kQ;         // key tiles, an item has two
  uint8_t K[kSlots][kTile];
  uint8_t Q[kQ][kTile];
  uint4 ones[256];          // the keys' channels for the log-sum-exps: cores of 8 rows x 16 bytes
  uint4 base[kTurns][256];  // the rows': -lse / scale in three parts; -inf: nobody's row
  int limit[kMeta][kTQ];    // positions that the row sees
  int unit[kMeta];
  float sum[2][kTK];        // of the second halves of the columns
  int ids[kPlaces][kTK / 16];  // page of each box of an item's keys
  uint64_t kfull[kSlots], kempty[kSlots], ufull[kMeta], qempty[kQ], uempty[kTurns], sfull[2][2], sempty[2][2], turn[2], summed[2][8], taken[2][8], placed[kPlaces], fin[2];
  uint32_t tmem;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x as the sum of three bf16 numbers, side by side.
__device__ __forceinline__ uint2 three_parts(float x) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(x);
  const float r = x - __bfloat162float(hi);
  const bool fine = r - r == 0.f;  // (an infinity has one part)
  const __nv_bfloat16 mid = __float2bfloat16_rn(fine ? r : 0.f);
  const __nv_bfloat16 lo = __float2bfloat16_rn(fine ? r - __bfloat162float(mid) : 0.f);
  const auto bits = [](__nv_bfloat16 y) { return (uint32_t)__bfloat16_as_ushort(y); };
  return make_uint2(bits(hi) | bits(mid) << 16, bits(lo));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) mass_tc_kernel(const __grid_constant__ CUtensorMap mapK,
                                                             const __grid_constant__ CUtensorMap mapQ, const MassArgs a,
                                                             int32_t* st) {
  using S = Smem<D>;
  extern __shared__ __align__(1024) uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      tc::mbar_init(&sm.kfull[i], 1);
      tc::mbar_init(&sm.kempty[i], 2);
    }
    for (int i = 0; i < kMeta; ++i) tc::mbar_init(&sm.ufull[i], 1);
    for (int i = 0; i < S::kQ; ++i) tc::mbar_init(&sm.qempty[i], 1);
    for (int i = 0; i < kTurns; ++i) {
      tc::mbar_init(&sm.uempty[i], 1);
      tc::mbar_init(&sm.sfull[i >> 1][i & 1], 2);  // the products, and who has seen the unit's description
      tc::mbar_init(&sm.sempty[i >> 1][i & 1], kWeights / 2);
    }
    for (int i = 0; i < 16; ++i) {
      tc::mbar_init(&sm.summed[i >> 3][i & 7], 1);
      tc::mbar_init(&sm.taken[i >> 3][i & 7], 1);
    }
    for (int i = 0; i < kPlaces; ++i) tc::mbar_init(&sm.placed[i], 1);
    tc::mbar_init(&sm.turn[0], 1);
    tc::mbar_init(&sm.turn[1], 1);
    tc::mbar_init(&sm.fin[0], 1);
    tc::mbar_init(&sm.fin[1], 1);
    tc::fence_mbar_init();
  }
  if (tid < 256) sm.ones[tid] = tid & 8 ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
  tc::fence_proxy_async_smem();
  if (warp == kKeys && lane == 0) {
    tc::prefetch_tensormap(&mapK);
    tc::prefetch_tensormap(&mapQ);
  }
  pdl_wait();
  const bool odd = (tc::smem_u32(raw) & 1023u) != 0;  // (the products' tiles lie on 1024 bytes)
  if (odd && tid == 0) status_set(st, FASTAR_ERR_CUDA);
  const bool stopped = odd || (tid == 0 && status_bad(st));
  if (warp == kProducts) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  // the warps that follow the items find their place
  MassWalk<kTK> walk;
  unsigned items = 0;
  int parts = 1;
  bool ok = true;
  {
    int most;
    items = walk.count(a, most, ok);
    if (!ok && tid == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    if (!ok) items = 0;
    parts = mass_parts(a, items, most, kTQ);
  }
  tc::tc_fence_before();
  const int stop = __syncthreads_or(stopped);
  tc::tc_fence_after();
  if (stop) {
    if (warp == kProducts) tc::tmem_dealloc(sm.tmem, 512);
    return;
  }
  const uint32_t tmem = sm.tmem;
  ok = true;
  bool bad = false;
  // (items that are not cut are G apart)
  const int by_tiles = (int)gridDim.x / a.H, by_heads = (int)gridDim.x - by_tiles * a.H;
  auto item = [&](unsigned it) -> const MassItem& {
    return parts > 1 ? walk.find(a, it / parts) : walk.next(a, it, gridDim.x, by_tiles, by_heads);
  };

  if (warp == kKeys) {
    // ================================================= keys
    const int box = min(1 << a.page_shift, 128);
    unsigned slot = 0, round = 0, count = 0;
    // an item's place and page ids are read one item ahead
    MassItem next;
    int next_id = -1;
    auto look = [&](unsigned it) {
      if (it >= items * parts) return;
      next = item(it);
      const int p = next.k0 + lane * box;
      next_id = lane * box < min(kTK, next.len - next.k0) ? a.table[(size_t)next.b * a.max_pages + (p >> a.page_shift)] : -1;
    };
    look(blockIdx.x);
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x, ++count) {
      const MassItem x = next;
      int id = next_id;
      look(it + gridDim.x);
      int t0, t1;
      mass_share(mass_tiles(a, x.n - x.i0, kTQ), it % parts, parts, t0, t1);
      if (t0 == t1) continue;
      const int p = x.k0 + lane * box;
      if (lane * box < min(kTK, x.len - x.k0) && (id < 0 || id >= a.n_pages)) {
        bad = true;
        id = -1;
      }
      bool told = parts > 1;  // (the masses of cut items are the join's)
      for (int j = 0; j < (x.len - x.k0 > 128 ? 2 : 1) && ok; ++j) {
        if (round > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.kempty[slot], (round - 1) & 1u));
        if (!ok) break;
        if (!told) {
          if (lane * box < kTK) sm.ids[count % kPlaces][lane] = id;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.placed[count % kPlaces]);
          told = true;
        }
        const bool mine = id >= 0 && (lane * box) >> 7 == j;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box * D * 2;
        if (lane == 0) tc::mbar_arrive_expect_tx(&sm.kfull[slot], bytes);
        __syncwarp();
        if (mine) {
          const int row = ((id * a.H + x.h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
          uint8_t* dst = sm.K[slot] + (lane * box & 127) * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tc::tma_load_2d(dst + c * 128 * 128, &mapK, &sm.kfull[slot], c * 64, row);
        }
        if (++slot == S::kSlots) {
          slot = 0;
          ++round;
        }
      }
    }
    // the copies have landed before the CTA exits, also when nobody takes them
    for (unsigned i = 0; i < S::kSlots; ++i) {
      const unsigned n = round + (i < slot);
      if (n && !tc::mbar_wait(&sm.kfull[i], (n - 1) & 1u)) ok = false;
    }
  } else if (warp == kProducts || warp == kProducts + 1) {
    // ================================================= products
    const int me = warp - kProducts;
    unsigned u = 0, slot = 0, phase = 0;  // of the item: first unit, first key tile
    bool issued = false;
    const uint64_t ones = tc::sdesc_kmajor_plain(tc::smem_u32(sm.ones), 128, 256);
    const uint32_t k0 = tc::smem_u32(sm.K), dS = tmem + me * 256;
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x) {
      const MassItem& x = item(it);
      int t0, t1;
      mass_share(mass_tiles(a, x.n - x.i0, kTQ), it % parts, parts, t0, t1);
      const int units = max(1, t1 - t0), tiles = t0 == t1 ? 0 : x.len - x.k0 > 128 ? 2 : 1;
      const unsigned slot1 = slot + 1 == S::kSlots ? 0 : slot + 1, phase1 = slot + 1 == S::kSlots ? phase ^ 1u : phase;
      // (also where none of its units is this warp's: it sees every phase)
      if (tiles > 0) ok = tc::mbar_wait(&sm.kfull[slot], phase);
      bool both = tiles < 2;
      ok = __all_sync(0xffffffffu, ok);
      int k = (int)(u + me & 1);
      const bool none = k >= units;
      for (; k < units && ok; k += 2) {
        const unsigned n = u + k;
        const uint32_t back = ((n >> 1) - 1) & 1u;  // parity of the weights of unit n - 2
        if (n >= 2) ok = tc::mbar_wait(&sm.sempty[me][0], back) && tc::mbar_wait(&sm.sempty[me][1], back);
        ok = ok && tc::mbar_wait(&sm.ufull[n % kMeta], (n / kMeta) & 1u);
        const int cols = sm.unit[n % kMeta] & 255;
        const uint32_t idesc = tc::idesc_bf16_f32(128, (cols + 15) & ~15, 0, 0);
        const int q = n % S::kQ;
        const uint32_t qd = tc::desc_low(tc::smem_u32(sm.Q[q]), 16);
        const uint64_t base = tc::sdesc_kmajor_plain(tc::smem_u32(sm.base[n % kTurns]), 128, 256);
        if (!both) {
          ok = ok && tc::mbar_wait(&sm.kfull[slot1], phase1);
          both = true;
        }
        // The units' products go out one after the other: side by side each would
        // take as long as both.
        if (n > 0) ok = ok && tc::mbar_wait(&sm.turn[me], me ? (n >> 1) & 1u : back);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t kd = tc::desc_low(k0 + (j ? slot1 : slot) * S::kTile, 16);
          if (tc::elect_one()) {
            if (j < tiles) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                // (the other warp needs a while to begin)
                if (j == tiles - 1 && c == D / 32) tc::mbar_arrive(&sm.turn[me ^ 1]);
                const uint32_t off = ((c >> 2) * 128 * 128 + (c & 3) * 32) / 16;
                tc::mma_bf16_low(dS + j * 128, kd + off, qd + off, idesc, c > 0 ? 1u : 0u);
              }
              // (the largest term last: it is rounded once)
              tc::mma_bf16(dS + j * 128, ones, base, idesc, 1u);
              if (k + 2 >= units) tc::mma_commit(&sm.kempty[j ? slot1 : slot]);
            }
            tc::mma_commit(&sm.sfull[me][j]);
            tc::mbar_arrive(&sm.sfull[me][j]);
            if (j == 1) {
              tc::mma_commit(&sm.qempty[q]);
              tc::mma_commit(&sm.uempty[n % kTurns]);
            }
          }
          __syncwarp();
        }
        if (tiles == 0 && lane == 0) tc::mbar_arrive(&sm.turn[me ^ 1]);
        issued = true;
      }
      if (!both) ok = ok && tc::mbar_wait(&sm.kfull[slot1], phase1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (none && lane == 0) {
        if (tiles > 0) tc::mbar_arrive(&sm.kempty[slot]);
        if (tiles > 1) tc::mbar_arrive(&sm.kempty[slot1]);
      }
      u += units;
      for (int j = 0; j < tiles; ++j)
        if (++slot == S::kSlots) {
          slot = 0;
          phase ^= 1u;
        }
    }
    if (issued) {
      // every product has finished before TMEM is freed
      if (tc::elect_one()) tc::mma_commit(&sm.fin[me]);
      __syncwarp();
      if (!tc::mbar_wait(&sm.fin[me], 0)) ok = false;
    }
  } else if (warp >= kRows) {
    // ================================================= rows
    const unsigned me = warp - kRows;
    constexpr int per = D / 8;  // 16-byte pieces of a row
    unsigned u = 0, sent = 0;   // sent: one behind the last unit that the lane has sent for
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x) {
      const MassItem& x = item(it);
      const int tokens = x.n - x.i0, rows = tokens * a.g;
      const bool by_head = mass_by_head(a, tokens, kTQ);
      const int of_head = (tokens + kTQ - 1) / kTQ;
      int t0, t1;
      mass_share(mass_tiles(a, tokens, kTQ), it % parts, parts, t0, t1);
      const int units = max(1, t1 - t0);  // an empty part has a unit too, of no rows
      for (int t = (int)((me - u) % kTurns); t < units; t += kTurns) {
        const unsigned n = u + t;  // the unit
        const int ms = n % kMeta, q = n % S::kQ;
        // first row, of the item or of head `head`
        const int head = by_head ? (t0 + t) / of_head : 0, r0 = (by_head ? t0 + t - head * of_head : t0 + t) * kTQ;
        const int live = t1 > t0 ? min(kTQ, (by_head ? tokens : rows) - r0) : 0, padded = (live + 15) & ~15;
        const int first = x.i0 + (by_head ? r0 : r0 / a.g);  // first token, which sees the fewest keys
        const int sees = live ? branch_limit(first, x.n, x.len, a.block) : 0;
        bool masked = sees - x.k0 < min(x.len - x.k0, kTK);
        // rows e * 32 + lane: their place, log-sum-exp and limit
        uint32_t from[4];
        float lse[4];
        int limit[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e * 32 + lane;
          from[e] = 0xffffffffu;
          limit[e] = 0;
          if (r < live) {
            const int i = by_head ? r0 + r : (r0 + r) / a.g;
            const int of = x.h * a.g + (by_head ? head : (r0 + r) - i * a.g);
            const int at = a.rows ? a.rows[x.lo + x.i0 + i] : x.lo + x.i0 + i;
            if (at < 0 || at >= a.N)
              bad = true;
            else
              from[e] = (uint32_t)of * a.N + at;
            limit[e] = masked ? branch_limit(x.i0 + i, x.n, x.len, a.block) : x.len;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) lse[e] = from[e] != 0xffffffffu ? a.lse[from[e]] : -INFINITY;
        uint2 base[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (lse[e] == -INFINITY) {
            from[e] = 0xffffffffu;  // it adds nothing, whatever its query
            limit[e] = 0;
          }
          base[e] = three_parts(from[e] == 0xffffffffu ? -INFINITY : -lse[e] / a.scale);
          masked = masked || (e * 32 + lane < padded && limit[e] == 0);
        }
        masked = __any_sync(0xffffffffu, masked);
        // What goes beside the queries, once the products of unit n - 4 are done, the
        // last turn of this warp (which sees every phase of the barrier).
        ok = __all_sync(0xffffffffu, n < kTurns || tc::mbar_wait(&sm.uempty[n % kTurns], (n / kTurns - 1) & 1u));
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e * 32 + lane;
          if (r < padded) {
            uint4* const to = sm.base[n % kTurns] + (r >> 3) * 16 + (r & 7);
            to[0] = make_uint4(base[e].x, base[e].y, 0u, 0u);
            to[8] = make_uint4(0u, 0u, 0u, 0u);
            sm.limit[ms][r] = limit[e];
          }
        }
        if (lane == 0) sm.unit[ms] = live | (masked ? kMasked : 0);
        tc::fence_proxy_async_smem();
        __syncwarp();
        // The queries, once the products of unit n - kQ are done, the last one in
        // their place.  (The phase before it, unit n - 2 kQ's, is over: that unit is n -
        // 4 or older, and as odd or even as n - 4; the phase behind it is unit n's.)
        ok = __all_sync(0xffffffffu, n < S::kQ || tc::mbar_wait(&sm.qempty[q], (n / S::kQ - 1) & 1u));
        if (!ok) break;
        if (by_head) {
          // (a box past the branch's rows brings others': nobody's columns)
          if (lane == 0 && live) {
            tc::mbar_arrive_expect_tx(&sm.ufull[ms], kTQ * D * 2);
            const int y = (int)((uint32_t)(x.h * a.g + head) * a.N + x.lo + first);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tc::tma_load_2d(sm.Q[q] + c * 128 * 128, &mapQ, &sm.ufull[ms], c * 64, y);
            sent = n + 1;
          } else if (lane == 0) {
            tc::mbar_arrive(&sm.ufull[ms]);
          }
          continue;
        }
        const uint32_t q0 = tc::smem_u32(sm.Q[q]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e * 32 >= padded) break;
          for (int k = 0; k < 32; k += 32 / per) {
            const int r = k + lane / per, c = lane % per;
            const uint32_t src = __shfl_sync(0xffffffffu, from[e], r);
            const bool there = src != 0xffffffffu;
            tc::cp_async16(q0 + tc::sw128_offset(e * 32 + r, c, 128),
                           (const char*)a.q + (there ? (size_t)src * (D * 2) + c * 16 : 0), there ? 16u : 0u);
          }
        }
        tc::cp_async_wait_all();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.ufull[ms]);
      }
      u += units;
    }
    tc::cp_async_wait_all();
    // the copies have landed before the CTA exits, also when nobody takes them
    if (sent && !tc::mbar_wait(&sm.ufull[(sent - 1) % kMeta], ((sent - 1) / kMeta) & 1u)) ok = false;
  } else {
    // ================================================= weights
    const int half = warp >> 3, tile = (warp >> 2) & 1, key = (warp & 7) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + tile * 128 + half * 64;
    const float scale2 = a.scale * kLog2e;
    unsigned u = 0, count = 0;
    unsigned shared = 0;  // items so far that both halves have columns of
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x, ++count) {
      const MassItem& x = item(it);
      const int tokens = x.n - x.i0;
      int t0, t1;
      mass_share(mass_tiles(a, tokens, kTQ), it % parts, parts, t0, t1);
      const int units = max(1, t1 - t0);
      const bool both = units > 1 || (t1 > t0 && min(kTQ, mass_by_head(a, tokens, kTQ) ? tokens : tokens * a.g - t0 * kTQ) > 64);
      const int p = x.k0 + key;  // (behind the branch's end nothing is done with it)
      int row = -1;
      float old = 0.f;
      if (half == 0 && parts == 1) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.placed[count % kPlaces], (count / kPlaces) & 1u));
        if (!ok) break;
        const int id = sm.ids[count % kPlaces][key >> min(a.page_shift, 7)];
        if (key < x.len - x.k0 && id >= 0) row = ((id * a.H + x.h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
        if (row >= 0 && a.decay != 1.f) old = a.mass[row];
      }
      float sum[2] = {0.f, 0.f};
      for (int k = 0; k < units; ++k, ++u) {
        const int ms = u % kMeta, side = u & 1;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.sfull[side][tile], (u >> 1) & 1u));
        if (!ok) break;
        const int unit = sm.unit[ms];
        tc::tc_fence_after();
        const int cols = min(64, (((unit & 255) + 15) & ~15) - half * 64);
        if (cols > 0 && tile * 128 < x.len - x.k0) {
          const int* limit = sm.limit[ms] + half * 64;
          const uint32_t t = tl + side * 256;
          auto weigh = [&](uint32_t* raw, auto masked, int c) {
            float* const v = reinterpret_cast<float*>(raw);
#pragma unroll
            for (int i = 0; i < 16; i += 2) tc::mul2(v[i], v[i + 1], scale2, scale2);
            if (decltype(masked)::value) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const int4 l = *reinterpret_cast<const int4*>(limit + c + i);
                v[i] = p < l.x ? v[i] : -INFINITY;
                v[i + 1] = p < l.y ? v[i + 1] : -INFINITY;
                v[i + 2] = p < l.z ? v[i + 2] : -INFINITY;
                v[i + 3] = p < l.w ? v[i + 3] : -INFINITY;
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = ex2(v[i]);
            // (a tree: one long chain of sums would hold the next exponentials up)
#pragma unroll
            for (int o = 8; o > 1; o >>= 1)
#pragma unroll
              for (int i = 0; i < o; i += 2) tc::add2(v[i], v[i + 1], v[i + o], v[i + o + 1]);
            tc::add2(sum[0], sum[1], v[0], v[1]);
          };
          // 16 columns while the next 16 are on their way
          uint32_t v0[16], v1[16];
          tc::tmem_ld16_async(t, v0);
          if (unit == kTQ) {
            // every row and key: without a branch (two chunks of 4,680 tokens 234 -> 215 us)
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              tc::tmem_wait16(v0);
              tc::tmem_ld16_async(t + c + 16, v1);
              weigh(v0, std::false_type(), c);
              tc::tmem_wait16(v1);
              if (c == 0) tc::tmem_ld16_async(t + 32, v0);
              weigh(v1, std::false_type(), c + 16);
            }
          } else {
            for (int c = 0; c < cols; c += 32) {
              tc::tmem_wait16(v0);
              if (c + 16 < cols) tc::tmem_ld16_async(t + c + 16, v1);
              weigh(v0, std::true_type(), c);
              if (c + 16 >= cols) break;
              tc::tmem_wait16(v1);
              if (c + 32 < cols) tc::tmem_ld16_async(t + c + 32, v0);
              weigh(v1, std::true_type(), c + 16);
            }
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.sempty[side][tile]);
      }
      if (!ok) break;
      float drew = sum[0] + sum[1];
      if (both) {
        const int slot = shared & 1;
        if (half == 1) {
          if (shared >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.taken[slot][warp & 7], ((shared >> 1) - 1) & 1u));
          if (!ok) break;
          sm.sum[slot][key] = drew;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.summed[slot][warp & 7]);
        } else {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.summed[slot][warp & 7], (shared >> 1) & 1u));
          if (!ok) break;
          drew += sm.sum[slot][key];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.taken[slot][warp & 7]);
        }
        ++shared;
      }
      if (half == 1) continue;
      if (parts > 1) {
        a.part[(size_t)it * kTK + key] = drew;
      } else if (row >= 0) {
        const int past = x.len - x.n;
        if (p < past && a.decay == 1.f)
          atomicAdd(a.mass + row, drew);  // (nobody else's: the sum is old + drew, rounded once)
        else
          mass_write(a, x.b, past, x.len, p, row, old, drew);
      }
    }
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (!ok) status_set(st, FASTAR_ERR_TIMEOUT);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kProducts) tc::tmem_dealloc(tmem, 512);
  pdl_trigger();
}

template <int D>
int launch_t(const MassArgs& a, int32_t* st, cudaStream_t s) {
  CUtensorMap k, q;
  const uint32_t box = (1u << a.page_shift) < 128u ? (1u << a.page_shift) : 128u;
  const uint64_t rows = ((uint64_t)a.n_pages * a.H) << a.page_shift;
  // without pages nothing is loaded; the map then describes the queries
  int rc = make_tmap_bf16_2d(&k, rows ? a.K : a.q, rows ? rows : 1, D, box, 64);
  if (rc == FASTAR_OK) rc = make_tmap_bf16_2d(&q, a.q, (uint64_t)a.Hq * a.N, D, kTQ, 64);
  if (rc != FASTAR_OK) return rc;
  constexpr int smem = (int)sizeof(Smem<D>);
  static_assert(smem <= 227 * 1024, "shared memory");
  auto kernel = mass_tc_kernel<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      launch_pdl(kernel, dim3(a.G), dim3(kThreads), smem, s, k, q, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_tc");
  return FASTAR_OK;
}

}  // namespace

int launch_mass_tc(int D, MassArgs a, int32_t* st, cudaStream_t s) {
  a.G = kCtas;
  a.split = mass_split(a, kTQ);
  const int rc = D == 128 ? launch_t<128>(a, st, s) : launch_t<64>(a, st, s);
  return rc == FASTAR_OK && a.split ? launch_mass_join(kTK, kTQ, a, st, s) : rc;
}

}  // namespace fastar
