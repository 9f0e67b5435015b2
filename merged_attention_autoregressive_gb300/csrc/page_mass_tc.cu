// fastar_page_mass on the tensor cores (tcgen05 + TMEM, bf16).
//
// One persistent CTA per SM takes its items (page_mass.cuh), 256 keys by 128
// rows at a time.  The scores are taken transposed, S^T = K Q^T: a key is a TMEM
// lane and a row a column, so that a thread sums the weights of its key in a
// register, and nothing but 256 sums leaves an item.
//   warps 0-15   weights: warp w takes the keys of lane quarter w % 4 of key tile
//                w / 4 % 2, and half w / 8 of the columns;
//   warp 16      keys: a page box per lane and column half by TMA;
//   warp 17      products: two of M 128, N = the live rows, K = D per unit, into
//                one of two halves of TMEM;
//   warps 18-21  rows: two warps per query tile in turn gather the rows, their
//                log-sum-exps and limits, and at an item's begin the places and old
//                masses of its keys, ahead of the products.
// Waits are bounded: one that runs out sets the status word, and every warp
// leaves its loop by its own bounded waits.
#include <math.h>

#include "page_mass.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kTK = 256, kTQ = 128, kCtas = 152;
constexpr int kWeights = 16, kKeys = 16, kProducts = 17, kRows = 18, kThreads = 22 * 32;
constexpr int kMeta = 4;  // units described ahead: the rows' warps fill unit u + 4 only after unit u + 2's products, so after unit u's weights
constexpr float kLog2e = 1.4426950408889634f;

struct Unit {
  int flags;       // kFirst, kLast of the item; kMasked: some row does not see every key; kEnd: none
  int cols;        // live rows
  int keys;        // live keys of the item
  int k0, past, born;
  int slot;        // of the item's rows, old masses and sums
  int part;        // of the workspace, -1: the item is whole
};
constexpr int kFirst = 1, kLast = 2, kMasked = 4, kEnd = 8;

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;       // bytes of 128 keys or rows
  static constexpr int kSlots = D == 128 ? 2 : 4; // items' keys
  uint8_t K[kSlots][2][kTile];
  uint8_t Q[2][kTile];
  float base[kMeta][kTQ];   // -lse log2 e; -inf: nobody's row
  int limit[kMeta][kTQ];    // positions that the row sees
  Unit unit[kMeta];
  int row[kMeta][kTK];      // place in the pages; -1: none
  float old[kMeta][kTK];
  float sum[kMeta][kTK];    // of the second half of the columns
  uint64_t kfull[kSlots], kempty[kSlots], ufull[kMeta], qempty[2], sfull[2], sempty[2], summed[kMeta][8], fin;
  uint32_t tmem;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) mass_tc_kernel(const __grid_constant__ CUtensorMap mapK, const MassArgs a,
                                                             int32_t* st) {
  using S = Smem<D>;
  extern __shared__ __align__(1024) uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      tc::mbar_init(&sm.kfull[i], 1);
      tc::mbar_init(&sm.kempty[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) {
      tc::mbar_init(&sm.ufull[i], 2);
      for (int k = 0; k < 8; ++k) tc::mbar_init(&sm.summed[i][k], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.qempty[i], 1);
      tc::mbar_init(&sm.sfull[i], 1);
      tc::mbar_init(&sm.sempty[i], kWeights);
    }
    tc::mbar_init(&sm.fin, 1);
    tc::fence_mbar_init();
  }
  if (warp == kKeys && lane == 0) tc::prefetch_tensormap(&mapK);
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
  if (warp == kKeys || warp >= kRows) {
    int most;
    items = walk.count(a, most, ok);
    if (!ok && lane == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
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

  if (warp == kKeys) {
    // ================================================= keys
    const int box = min(1 << a.page_shift, 128);
    unsigned slot = 0, round = 0;
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x) {
      const MassItem x = walk.find(a, it / parts);
      const int tiles = (x.rows + kTQ - 1) / kTQ, part = it % parts;
      if ((long long)tiles * part / parts == (long long)tiles * (part + 1) / parts) continue;
      const int p = x.k0 + lane * box;
      int id = -1;
      if (lane * box < min(kTK, x.len - x.k0)) {
        id = a.table[(size_t)x.b * a.max_pages + (p >> a.page_shift)];
        if (id < 0 || id >= a.n_pages) {
          bad = true;
          id = -1;
        }
      }
      if (round > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.kempty[slot], (round - 1) & 1u));
      if (!ok) break;
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, id >= 0)) * box * D * 2;
      if (lane == 0) tc::mbar_arrive_expect_tx(&sm.kfull[slot], bytes);
      __syncwarp();
      if (id >= 0) {
        const int at = lane * box, row = ((id * a.H + x.h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
        uint8_t* dst = sm.K[slot][at >> 7] + (at & 127) * 128;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tc::tma_load_2d(dst + c * 128 * 128, &mapK, &sm.kfull[slot], c * 64, row);
      }
      if (++slot == S::kSlots) {
        slot = 0;
        ++round;
      }
    }
    // the copies have landed before the CTA exits, also when nobody takes them
    for (unsigned i = 0; i < S::kSlots; ++i) {
      const unsigned n = round + (i < slot);
      if (n && !tc::mbar_wait(&sm.kfull[i], (n - 1) & 1u)) ok = false;
    }
  } else if (warp == kProducts) {
    // ================================================= products
    unsigned slot = 0, kphase = 0;
    bool issued = false;
    for (unsigned u = 0; ok; ++u) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.ufull[u % kMeta], (u / kMeta) & 1u));
      if (!ok) break;
      const Unit d = sm.unit[u % kMeta];
      if (d.flags & kEnd) break;
      if (u >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.sempty[u & 1], ((u >> 1) - 1) & 1u));
      if (ok && (d.flags & kFirst) && d.cols) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.kfull[slot], kphase));
      if (!ok) break;
      tc::tc_fence_after();
      const int n = (d.cols + 15) & ~15;
      const uint32_t idesc = tc::idesc_bf16_f32(128, n, 0, 0);
      const uint32_t kd = tc::desc_low(tc::smem_u32(sm.K[slot][0]), 16), qd = tc::desc_low(tc::smem_u32(sm.Q[u & 1]), 16);
      const uint32_t dS = tmem + (u & 1) * 256;
      const int two = d.keys > 128 ? 2 : 1;
      if (tc::elect_one()) {
        if (d.cols) {
          for (int j = 0; j < two; ++j)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * 128 * 128 + (k & 3) * 32) / 16;
              tc::mma_bf16_low(dS + j * 128, kd + j * (S::kTile / 16) + off, qd + off, idesc, k > 0 ? 1u : 0u);
            }
        }
        tc::mma_commit(&sm.qempty[u & 1]);
        tc::mma_commit(&sm.sfull[u & 1]);
        if ((d.flags & kLast) && d.cols) tc::mma_commit(&sm.kempty[slot]);
      }
      __syncwarp();
      issued = true;
      if ((d.flags & kLast) && d.cols && ++slot == S::kSlots) {
        slot = 0;
        kphase ^= 1u;
      }
    }
    if (issued) {
      // every product has finished before TMEM is freed
      if (tc::elect_one()) tc::mma_commit(&sm.fin);
      __syncwarp();
      if (!tc::mbar_wait(&sm.fin, 0)) ok = false;
    }
  } else if (warp >= kRows) {
    // ================================================= rows
    const int group = (warp - kRows) >> 1, half = (warp - kRows) & 1;
    constexpr int per = D / 8;  // 16-byte pieces of a row
    unsigned u = 0, count = 0;
    for (unsigned it = blockIdx.x; it < items * parts && ok; it += gridDim.x, ++count) {
      const MassItem x = walk.find(a, it / parts);
      const int tiles = (x.rows + kTQ - 1) / kTQ, part = it % parts;
      const int t0 = (int)((long long)tiles * part / parts), t1 = (int)((long long)tiles * (part + 1) / parts);
      const int units = max(1, t1 - t0);  // an empty part has a unit too, of no rows
      for (int t = 0; t < units; ++t, ++u) {
        if ((int)(u & 1) != group) continue;
        if (u >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.qempty[group], ((u >> 1) - 1) & 1u));
        if (!ok) break;
        const int ms = u % kMeta, slot = count % kMeta;
        const int r0 = (t0 + t) * kTQ, live = t1 > t0 ? min(kTQ, x.rows - r0) : 0, padded = (live + 15) & ~15;
        // two rows per lane: their place, log-sum-exp and limit
        uint32_t from[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = half * 64 + e * 32 + lane;
          from[e] = 0xffffffffu;
          float base = -INFINITY;
          int limit = 0;
          if (r < live) {
            const int i = (r0 + r) / a.g, head = x.h * a.g + (r0 + r) - i * a.g;
            const int at = a.rows ? a.rows[x.lo + x.i0 + i] : x.lo + x.i0 + i;
            if (at < 0 || at >= a.N) {
              bad = true;
            } else {
              const uint32_t y = (uint32_t)head * a.N + at;
              const float lse = a.lse[y];
              if (lse != -INFINITY) {
                from[e] = y;
                base = -lse * kLog2e;
                limit = mass_limit(x.i0 + i, x.n, x.len, a.block);
              }
            }
          }
          if (r < padded) {
            sm.base[ms][r] = base;
            sm.limit[ms][r] = limit;
          }
        }
        // their queries, 16 bytes per lane
        const uint32_t q0 = tc::smem_u32(sm.Q[group]);
        const int end = min(64, padded - half * 64);
        for (int k = 0; k < end; k += 32 / per) {
          const int r = k + lane / per, c = lane % per;
          const uint32_t src = __shfl_sync(0xffffffffu, k & 32 ? from[1] : from[0], r & 31);
          const bool there = src != 0xffffffffu;
          tc::cp_async16(q0 + tc::sw128_offset(half * 64 + r, c, 128),
                         (const char*)a.q + (there ? (size_t)src * (D * 2) + c * 16 : 0), there ? 16u : 0u);
        }
        if (t == 0) {
          // the item's keys: four per lane
          int row[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = (half * 4 + e) * 32 + lane;
            row[e] = k < x.len - x.k0 ? mass_row(a, x.b, x.h, x.k0 + k) : -1;
            bad = bad || (k < x.len - x.k0 && row[e] < 0);
          }
          float old[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) old[e] = row[e] >= 0 && parts == 1 ? a.mass[row[e]] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sm.row[slot][(half * 4 + e) * 32 + lane] = row[e];
            sm.old[slot][(half * 4 + e) * 32 + lane] = old[e];
          }
        }
        if (half == 0 && lane == 0) {
          Unit d;
          // the tile's first row sees the fewest keys
          const int first = live ? mass_limit(x.i0 + r0 / a.g, x.n, x.len, a.block) : 0;
          d.flags = (t == 0 ? kFirst : 0) | (t == units - 1 ? kLast : 0) | (first - x.k0 < min(x.len - x.k0, kTK) ? kMasked : 0);
          d.cols = live;
          d.keys = x.len - x.k0;
          d.k0 = x.k0;
          d.past = x.len - x.n;
          d.born = a.born ? a.total[x.b] - x.len : 0;
          d.slot = slot;
          d.part = parts > 1 ? (int)it : -1;
          sm.unit[ms] = d;
        }
        tc::cp_async_wait_all();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.ufull[ms]);
      }
    }
    // no unit: the end (the group whose turn it is)
    if (ok && (int)(u & 1) == group) {
      if (u >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.qempty[group], ((u >> 1) - 1) & 1u));
      if (ok && lane == 0) {
        if (half == 0) sm.unit[u % kMeta].flags = kEnd;
        tc::mbar_arrive(&sm.ufull[u % kMeta]);
      }
    }
    tc::cp_async_wait_all();
  } else {
    // ================================================= weights
    const int tile = (warp >> 2) & 1, half = warp >> 3;
    const int key = tile * 128 + (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + tile * 128 + half * 64;
    const float scale2 = a.scale * kLog2e;
    float sum[8];
    unsigned count = 0;
    for (unsigned u = 0; ok; ++u) {
      const int ms = u % kMeta;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.ufull[ms], (u / kMeta) & 1u));
      if (!ok) break;
      const Unit d = sm.unit[ms];
      if (d.flags & kEnd) break;
      if (d.flags & kFirst) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
      }
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.sfull[u & 1], (u >> 1) & 1u));
      if (!ok) break;
      tc::tc_fence_after();
      const int cols = min(64, ((d.cols + 15) & ~15) - half * 64);
      if (tile * 128 < d.keys) {
        const uint32_t t = tl + (u & 1) * 256;
        const float* base = sm.base[ms] + half * 64;
        const int* limit = sm.limit[ms] + half * 64;
        const int p = d.k0 + key;
        int c = 0;
        for (; c + 32 <= cols; c += 32) {
          float v[32];
          tc::tmem_ld32(t + c, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 b = *reinterpret_cast<const float4*>(base + c + i);
            tc::fma2(v[i], v[i + 1], scale2, scale2, b.x, b.y);
            tc::fma2(v[i + 2], v[i + 3], scale2, scale2, b.z, b.w);
          }
          if (d.flags & kMasked) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int4 l = *reinterpret_cast<const int4*>(limit + c + i);
              v[i] = p < l.x ? v[i] : -INFINITY;
              v[i + 1] = p < l.y ? v[i + 1] : -INFINITY;
              v[i + 2] = p < l.z ? v[i + 2] : -INFINITY;
              v[i + 3] = p < l.w ? v[i + 3] : -INFINITY;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) tc::add2(sum[i & 7], sum[(i & 7) + 1], ex2(v[i]), ex2(v[i + 1]));
        }
        for (; c < cols; c += 8) {
          float v[8];
          tc::tmem_ld8(t + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sum[i] += p < limit[c + i] ? ex2(fmaf(v[i], scale2, base[c + i])) : 0.f;
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.sempty[u & 1]);
      if (d.flags & kLast) {
        float drew = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
        const int pair = warp & 7;
        // the second half's sums; a slot is free again two units later
        if (half == 1) {
          sm.sum[d.slot][key] = drew;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.summed[d.slot][pair]);
        } else {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.summed[d.slot][pair], (count / kMeta) & 1u));
          if (!ok) break;
          drew += sm.sum[d.slot][key];
          const int row = sm.row[d.slot][key], p = d.k0 + key;
          if (d.part >= 0) {
            a.part[(size_t)d.part * kTK + key] = drew;
          } else if (row >= 0) {
            a.mass[row] = p >= d.past ? drew : fmaf(a.decay, sm.old[d.slot][key], drew);
            if (a.born && p >= d.past) a.born[row] = d.born + p;
          }
        }
        ++count;
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
  CUtensorMap k;
  const uint32_t box = (1u << a.page_shift) < 128u ? (1u << a.page_shift) : 128u;
  const uint64_t rows = ((uint64_t)a.n_pages * a.H) << a.page_shift;
  // without pages nothing is loaded; the map then describes the queries
  const int rc = make_tmap_bf16_2d(&k, rows ? a.K : a.q, rows ? rows : 1, D, box, 64);
  if (rc != FASTAR_OK) return rc;
  constexpr int smem = (int)sizeof(Smem<D>);
  static_assert(smem <= 227 * 1024, "shared memory");
  auto kernel = mass_tc_kernel<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      launch_pdl(kernel, dim3(a.G), dim3(kThreads), smem, s, k, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_tc");
  return FASTAR_OK;
}

}  // namespace

int launch_mass_tc(int D, MassArgs a, int32_t* st, cudaStream_t s) {
  a.G = kCtas;
  // cut only where a branch may have rows for two tiles of them
  a.split = (long long)a.M * a.g > kTQ;
  const int rc = D == 128 ? launch_t<128>(a, st, s) : launch_t<64>(a, st, s);
  return rc == FASTAR_OK && a.split ? launch_mass_join(kTK, kTQ, a, st, s) : rc;
}

}  // namespace fastar
