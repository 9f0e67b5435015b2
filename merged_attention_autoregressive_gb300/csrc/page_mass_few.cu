// fastar_page_mass for branches of a few rows: single tokens, short drafts.
//
// bf16: the keys pass through once and nothing is done twice with them, so they go
// from memory straight into the registers of warp-level products (m 16 keys, n 8
// rows, k 16 channels): a warp takes 16 keys, lane 4 r + t the 16-byte pieces t, t +
// 4, ... of keys r and r + 8, and the same pieces of row r.  A piece is two steps'
// operands: which channel is which does not matter to a sum over all of them, as
// long as keys and rows agree.  A thread then holds the scores of two keys and two
// rows; their weights are summed over the rows by two shuffles.  No shared memory,
// no barrier, and as many loads in flight as warps fit.
//
// What bounds it: HBM.  16 single tokens of 40 heads over 4,681 keys: 117 us, 6.8 TB/s
// (by the tensor cores' kernel 147 us: an item's handovers take longer than its
// loads); a call of a few branches is a launch and four dependent reads, 4 us.
#include <math.h>

#include "page_mass.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kTK = 128, kThreads = 256, kPerSm = 3;
constexpr int kTK32 = 64, kThreads32 = 128;
constexpr int per_sm32(int D) { return D == 128 ? 3 : 4; }  // (4 of 128 channels spill: single tokens 75 us for 70)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) mass_few_kernel(const MassArgs a, int32_t* st) {
  pdl_wait();
  if (block_status_bad(st)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  constexpr int kPieces = D / 32;  // 16-byte pieces of a key that a lane takes
  const float scale2 = a.scale * kLog2e;
  MassWalk<kTK> walk;
  int most;
  bool ok = true, bad = false;
  const unsigned items = walk.count(a, most, ok);
  if (!ok) {
    if (threadIdx.x == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    return;
  }
  const int by_tiles = (int)gridDim.x / a.H, by_heads = (int)gridDim.x - by_tiles * a.H;
  // the page ids of the lane's two keys are read one item ahead
  int id[2] = {-1, -1};
  MassItem y = {};
  auto look = [&](unsigned it) {
    if (it >= items) return;
    y = walk.next(a, it, gridDim.x, by_tiles, by_heads);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = warp * 16 + r + 8 * e;
      id[e] = k < y.len - y.k0 ? a.table[(size_t)y.b * a.max_pages + ((y.k0 + k) >> a.page_shift)] : -2;
    }
  };
  look(blockIdx.x);
  for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {
    const MassItem x = y;
    int row[2];
    uint4 key[2][kPieces];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int p = x.k0 + warp * 16 + r + 8 * e;
      row[e] = -1;
      if (id[e] >= 0 && id[e] < a.n_pages)
        row[e] = ((id[e] * a.H + x.h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
      else if (id[e] != -2)
        bad = true;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        key[e][j] = make_uint4(0u, 0u, 0u, 0u);
        if (row[e] >= 0) key[e][j] = __ldcs(reinterpret_cast<const uint4*>((const char*)a.K + (size_t)row[e] * (D * 2)) + t + 4 * j);
      }
    }
    look(it + gridDim.x);
    if (!__any_sync(0xffffffffu, row[0] >= 0)) continue;  // (the rows come in order: no key of the warp's is there)
    const int at = t == 0 ? row[0] : t == 1 ? row[1] : -1;  // lane t = 0, 1 of a key's four writes the mass of key r, r + 8
    const float old = at >= 0 ? a.mass[at] : 0.f;
    const int rows = x.n * a.g;
    float drew[2] = {0.f, 0.f};
    for (int r0 = 0; r0 < rows; r0 += 8) {
      // the queries of row r0 + r, and what belongs to the scores' rows r0 + 2 t + e
      auto place = [&](int i) -> long long {  // of row i in q and lse
        if (i >= rows) return -1;
        const int token = i / a.g, head = x.h * a.g + i - token * a.g;
        const int n = a.rows ? a.rows[x.lo + token] : x.lo + token;
        if (n < 0 || n >= a.N) {
          bad = true;
          return -1;
        }
        return (long long)head * a.N + n;
      };
      const long long from = place(r0 + r);
      uint4 query[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        query[j] = make_uint4(0u, 0u, 0u, 0u);
        if (from >= 0) query[j] = *(reinterpret_cast<const uint4*>((const char*)a.q + (size_t)from * (D * 2)) + t + 4 * j);
      }
      float base[2];
      int limit[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = r0 + 2 * t + e;
        const long long f = place(i);
        const float lse = f >= 0 ? a.lse[f] : -INFINITY;
        base[e] = -lse * kLog2e;
        limit[e] = lse == -INFINITY ? 0 : branch_limit(i / a.g, x.n, x.len, a.block);
      }
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        mma_16816(c, key[0][j].x, key[1][j].x, key[0][j].y, key[1][j].y, query[j].x, query[j].y);
        mma_16816(c, key[0][j].z, key[1][j].z, key[0][j].w, key[1][j].w, query[j].z, query[j].w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (warp * 16 + r + 8 * k < limit[e] - x.k0) drew[k] += ex2(fmaf(c[2 * k + e], scale2, base[e]));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      drew[k] += __shfl_xor_sync(0xffffffffu, drew[k], 1);
      drew[k] += __shfl_xor_sync(0xffffffffu, drew[k], 2);
    }
    if (at >= 0)
      mass_write(a, x.b, x.len - x.n, x.len, x.k0 + warp * 16 + r + 8 * t, at, old, t == 0 ? drew[0] : drew[1]);
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  pdl_trigger();
}

// The same in 32 bits, on the FP32 pipes: eight lanes share a key, lane t its 16-byte
// pieces t, t + 8, ..., and hold four keys each; two rows at a time come out of L1, and
// the partial sums of four keys and two rows are added over the eight lanes so that
// each ends with the score of one key and one row.
//
// What bounds it: HBM for single tokens (16 of 12 heads over 4,681 keys: 70 us, 6.7
// TB/s, by the kernel for many rows 202 us; D 64 40 and 122 us), reads of rows and
// shuffles for more (16 tokens a branch 164 and 231 us, 32 tokens 287 and 278 us).
template <int D>
__global__ void __launch_bounds__(kThreads32, per_sm32(D)) mass_few32_kernel(const MassArgs a, int32_t* st) {
  pdl_wait();
  if (block_status_bad(st)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 3, t = lane & 7;
  constexpr int kPieces = D / 32, kKeys = 4;  // 16-byte pieces of a key that a lane takes, and its keys
  const float scale2 = a.scale * kLog2e;
  MassWalk<kTK32> walk;
  int most;
  bool ok = true, bad = false;
  const unsigned items = walk.count(a, most, ok);
  if (!ok) {
    if (threadIdx.x == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    return;
  }
  const int by_tiles = (int)gridDim.x / a.H, by_heads = (int)gridDim.x - by_tiles * a.H;
  // the page ids of the lane's keys, warp * 16 + r + 4 e, are read one item ahead
  int id[kKeys];
  MassItem y = {};
  auto look = [&](unsigned it) {
    if (it >= items) return;
    y = walk.next(a, it, gridDim.x, by_tiles, by_heads);
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      const int k = warp * 16 + r + 4 * e;
      id[e] = k < y.len - y.k0 ? a.table[(size_t)y.b * a.max_pages + ((y.k0 + k) >> a.page_shift)] : -2;
    }
  };
  look(blockIdx.x);
  for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {
    const MassItem x = y;
    const int p0 = x.k0 + warp * 16 + r;
    int mine = -1;  // the row of the lane's own key, whose score it gets
    float4 key[kKeys][kPieces];
    const int own = 2 * (t & 1) + (t >> 1 & 1);
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      int row = -1;
      if (id[e] >= 0 && id[e] < a.n_pages)
        row = ((id[e] * a.H + x.h) << a.page_shift) + ((p0 + 4 * e) & ((1 << a.page_shift) - 1));
      else if (id[e] != -2)
        bad = true;
      if (e == own) mine = row;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        key[e][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) key[e][j] = __ldcs(reinterpret_cast<const float4*>((const float*)a.K + (size_t)row * D) + t + 8 * j);
      }
    }
    look(it + gridDim.x);
    if (x.k0 + warp * 16 >= x.len) continue;  // (no key of the warp's is there)
    const int p = p0 + 4 * own;
    const int end = (x.n - x.i0) * a.g;
    const float old = mine >= 0 && t < 4 ? a.mass[mine] : 0.f;
    float drew = 0.f;
    for (int i0 = 0; i0 < end; i0 += 32) {
      // a row per lane: its place in q, its log-sum-exp, the positions that it sees
      int from = -1, limit = 0;
      float base = 0.f;
      if (i0 + lane < end) {
        const int token = x.i0 + (i0 + lane) / a.g, head = x.h * a.g + (i0 + lane) % a.g;
        const int at = a.rows ? a.rows[x.lo + token] : x.lo + token;
        if (at < 0 || at >= a.N) {
          bad = true;
        } else {
          const float lse = a.lse[(size_t)head * a.N + at];
          if (lse != -INFINITY) {
            from = head * a.N + at;
            base = -lse * kLog2e;
            limit = branch_limit(token, x.n, x.len, a.block);
          }
        }
      }
      const int n = min(32, end - i0);
      for (int i = 0; i < n; i += 2) {
        float s[2][kKeys], s1[2][kKeys];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int f = __shfl_sync(0xffffffffu, from, i + w);  // (i + 1 <= 31)
          float4 q[kPieces];
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            q[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (f >= 0) q[j] = *(reinterpret_cast<const float4*>((const float*)a.q + (size_t)f * D) + t + 8 * j);
          }
#pragma unroll
          for (int e = 0; e < kKeys; ++e) {
            s[w][e] = s1[w][e] = 0.f;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
              tc::fma_pair(s[w][e], s1[w][e], q[j].x, q[j].y, key[e][j].x, key[e][j].y);
              tc::fma_pair(s[w][e], s1[w][e], q[j].z, q[j].w, key[e][j].z, key[e][j].w);
            }
            s[w][e] += s1[w][e];
          }
        }
        // the eight lanes of a key add up, and share out keys and rows
        float v[2];
        const bool b0 = t & 1, b1 = t & 2, b2 = t & 4;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float u0 = (b0 ? s[w][2] : s[w][0]) + __shfl_xor_sync(0xffffffffu, b0 ? s[w][0] : s[w][2], 1);
          const float u1 = (b0 ? s[w][3] : s[w][1]) + __shfl_xor_sync(0xffffffffu, b0 ? s[w][1] : s[w][3], 1);
          v[w] = (b1 ? u1 : u0) + __shfl_xor_sync(0xffffffffu, b1 ? u0 : u1, 2);
        }
        const float score = (b2 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, b2 ? v[0] : v[1], 4);
        const float off = __shfl_sync(0xffffffffu, base, i + (t >> 2));
        const int lim = __shfl_sync(0xffffffffu, limit, i + (t >> 2));
        if (p < lim) drew += exp2f(fmaf(score, scale2, off));
      }
    }
    drew += __shfl_xor_sync(0xffffffffu, drew, 4);
    if (t < 4 && mine >= 0) mass_write(a, x.b, x.len - x.n, x.len, p, mine, old, drew);
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  pdl_trigger();
}

}  // namespace

int launch_mass_few(int D, bool bf16, MassArgs a, int32_t* st, cudaStream_t s) {
  auto kernel = bf16 ? D == 128 ? mass_few_kernel<128> : mass_few_kernel<64>
                     : D == 128 ? mass_few32_kernel<128> : mass_few32_kernel<64>;
  const int ctas = 152 * (bf16 ? kPerSm : per_sm32(D));
  if (launch_pdl(kernel, dim3(ctas), dim3(bf16 ? kThreads : kThreads32), 0, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_few");
  return FASTAR_OK;
}

}  // namespace fastar
