// fastar_page_mass for branches of a few rows (bf16): single tokens, short drafts.
//
// The keys pass through once and nothing is done twice with them, so they go
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

}  // namespace

int launch_mass_few(int D, MassArgs a, int32_t* st, cudaStream_t s) {
  auto kernel = D == 128 ? mass_few_kernel<128> : mass_few_kernel<64>;
  if (launch_pdl(kernel, dim3(152 * kPerSm), dim3(kThreads), 0, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_few");
  return FASTAR_OK;
}

}  // namespace fastar
