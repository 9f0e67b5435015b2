// fastar_page_mass in 32 bits for branches of many rows, the join of cut items, and
// the dispatch.
//
// w(i, p) = exp(scale q_i . k_p - lse_i), summed over the rows i that see
// position p.  A CTA of 256 threads holds 64 keys and takes 64 rows at a time:
// 4 x 4 scores per thread, their weights added over the thread's four rows; at
// the item's end the sums of the 16 threads of a key are joined.  A thread's loads
// go out side by side (drafts of 9 branches, up to 24 tokens of 3 heads a group,
// D 64: 13.1 us; one after the other 17.3 us), three CTAs fit on an SM.
//
// What bounds it: latency where rows are few (that call: two items per CTA, each a
// chain of page id, key and row reads), reads of shared memory where they are many (64
// tokens of 16 branches, 12 heads over 4,744 keys: 436 us, of which the multiply-adds
// are 200 us; a 16-byte read takes a warp four cycles whatever its lanes share, so
// other places of a thread's scores gain nothing, and 8 x 4 of them 8 % of long calls
// for 5 to 60 % of short ones).
#include <math.h>

#include "page_mass.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kTK = 64, kTQ = 64, kThreads = 256, kPerSm = 3, kCtas = kPerSm * 152;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Smem {
  float K[kTK][D + 4];
  float Q[kTQ][D + 4];
  float base[kTQ];      // -lse log2 e
  int limit[kTQ];       // positions that the row sees; 0: none, or nobody's row
  long long from[kTQ];  // place in q; -1: its score does not matter
  int row[kTK];         // in the pages; -1: none
  float old[kTK];
  float sum[kThreads / 32][kTK];
};

template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) mass_simt_kernel(const MassArgs a, int32_t* st) {
  pdl_wait();
  extern __shared__ uint4 raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  if (block_status_bad(st)) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  constexpr int RV = D / 4;  // vectors of a row
  const float scale2 = a.scale * kLog2e;
  MassWalk<kTK> walk;
  int most;
  bool ok = true, bad = false;
  const unsigned items = walk.count(a, most, ok);
  if (!ok) {
    if (tid == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    return;
  }
  const int parts = mass_parts(a, items, most, kTQ);
  for (unsigned it = blockIdx.x; it < items * parts; it += gridDim.x) {
    const MassItem x = walk.find(a, it / parts);
    const int part = (int)(it % parts), rows = (x.n - x.i0) * a.g, tiles = mass_tiles(a, x.n - x.i0, kTQ);
    int t0, t1;
    mass_share(tiles, part, parts, t0, t1);
    // what belongs to the rows of tile t (64 threads)
    auto describe = [&](int r, int t) {
      const int i = t * kTQ + r;
      long long from = -1;
      float base = 0.f;
      int limit = 0;
      if (i < rows && t < t1) {
        const int token = x.i0 + i / a.g, head = x.h * a.g + i % a.g;
        const int at = a.rows ? a.rows[x.lo + token] : x.lo + token;
        if (at < 0 || at >= a.N) {
          bad = true;
        } else {
          const float lse = a.lse[(size_t)head * a.N + at];
          if (lse != -INFINITY) {
            from = (long long)head * a.N + at;
            base = -lse * kLog2e;
            limit = branch_limit(token, x.n, x.len, a.block);
          }
        }
      }
      sm.from[r] = from;
      sm.base[r] = base;
      sm.limit[r] = limit;
    };
    // 64 rows into shared memory, a thread's loads side by side
    constexpr int kLoads = kTK * RV / kThreads;
    auto fetch = [&](const float* src, auto place, float (*dst)[D + 4]) {
      float4 v[kLoads];
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int r = (e * kThreads + tid) / RV, c = (e * kThreads + tid) % RV;
        const long long at = place(r);
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at >= 0) v[e] = *(reinterpret_cast<const float4*>(src + (size_t)at * D) + c);
      }
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int r = (e * kThreads + tid) / RV, c = (e * kThreads + tid) % RV;
        *reinterpret_cast<float4*>(&dst[r][c * 4]) = v[e];
      }
    };
    if (tid < kTK) {
      int row = -1;
      if (tid < x.len - x.k0) {
        row = mass_row(a, x.b, x.h, x.k0 + tid);
        bad = bad || row < 0;
      }
      sm.row[tid] = row;
      sm.old[tid] = row >= 0 && parts == 1 ? a.mass[row] : 0.f;
    } else if (tid < kTK + kTQ) {
      describe(tid - kTK, t0);
    }
    __syncthreads();
    fetch((const float*)a.K, [&](int r) { return (long long)sm.row[r]; }, sm.K);
    float drew[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = t0; t < t1; ++t) {
      if (t > t0) {
        __syncthreads();
        if (tid < kTQ) describe(tid, t);
        __syncthreads();
      }
      const int live = min(kTQ, rows - t * kTQ);
      fetch((const float*)a.q, [&](int r) { return sm.from[r]; }, sm.Q);
      __syncthreads();
      if ((ty & ~1) * 4 >= live) continue;  // no row of the warp
      float s[4][4], s1[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = s1[i][j] = 0.f;
#pragma unroll 2
      for (int k = 0; k < D; k += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&sm.Q[ty * 4 + i][k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&sm.K[tx + 16 * j][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // even and odd channels have a sum each
            tc::fma_pair(s[i][j], s1[i][j], qv[i].x, qv[i].y, kv[j].x, kv[j].y);
            tc::fma_pair(s[i][j], s1[i][j], qv[i].z, qv[i].w, kv[j].z, kv[j].w);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float base = sm.base[ty * 4 + i];
        const int limit = sm.limit[ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tx + 16 * j < limit - x.k0) drew[j] += exp2f(fmaf(s[i][j] + s1[i][j], scale2, base));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      drew[j] += __shfl_xor_sync(0xffffffffu, drew[j], 16);
      if ((tid & 31) < 16) sm.sum[tid >> 5][tx + 16 * j] = drew[j];
    }
    __syncthreads();
    if (tid < kTK) {
      float d = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) d += sm.sum[w][tid];
      const int row = sm.row[tid];
      if (parts > 1)
        a.part[(size_t)it * kTK + tid] = d;
      else if (row >= 0)
        mass_write(a, x.b, x.len - x.n, x.len, x.k0 + tid, row, sm.old[tid], d);
    }
    __syncthreads();
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  pdl_trigger();
}

// Adds the parts of the items that are cut, in order; a CTA per item.
template <int TK, int TQ>
__global__ void __launch_bounds__(TK) mass_join_kernel(const MassArgs a, int32_t* st) {
  pdl_wait();
  if (block_status_bad(st)) return;
  MassWalk<TK> walk;
  int most;
  bool ok = true;
  const unsigned items = walk.count(a, most, ok);
  const int parts = ok ? mass_parts(a, items, most, TQ) : 1;
  if (parts == 1 || blockIdx.x >= items) return;
  const MassItem x = walk.find(a, blockIdx.x);
  if ((int)threadIdx.x >= x.len - x.k0) return;
  const int p = x.k0 + threadIdx.x;
  const int row = mass_row(a, x.b, x.h, p);
  if (row < 0) return;
  const float old = a.mass[row];
  float d = 0.f;
  for (int i = 0; i < parts; ++i) d += a.part[((size_t)blockIdx.x * parts + i) * TK + threadIdx.x];
  mass_write(a, x.b, x.len - x.n, x.len, p, row, old, d);
}

template <int D>
int launch_t(const MassArgs& a, int32_t* st, cudaStream_t s) {
  constexpr int smem = (int)sizeof(Smem<D>);
  auto kernel = mass_simt_kernel<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      launch_pdl(kernel, dim3(a.G), dim3(kThreads), smem, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_simt");
  return a.split ? launch_mass_join(kTK, kTQ, a, st, s) : FASTAR_OK;
}

}  // namespace

// Tiles of keys and rows as in the kernel that left the sums.
int launch_mass_join(int TK, int TQ, const MassArgs& a, int32_t* st, cudaStream_t s) {
  auto kernel = TK == 64 ? mass_join_kernel<64, 64> : mass_join_kernel<256, 128>;
  if (launch_pdl(kernel, dim3(a.G * kMostParts / 2), dim3(TK), 0, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_mass_join");
  return FASTAR_OK;
}

size_t mass_ws_bytes(int Hq, int H, int M, int D) {
  if (Hq < 1 || H < 1 || M < 1 || D < 1 || Hq % H) return 0;
  return (size_t)kMostParts * 152 * 256 * 4;  // (64-key tiles of three times the CTAs need less)
}

int launch_page_mass(const fastar_pages* pg, const void* q, const float* lse, int Hq, int N, const int32_t* rows,
                     int M, const int32_t* cu, float scale, int block, float decay, const fastar_mass* mass, void* ws,
                     int32_t* st, cudaStream_t s) {
  MassArgs a = {};
  a.q = q;
  a.lse = lse;
  a.rows = rows;
  a.cu = cu;
  a.len = pg->len;
  a.table = pg->table;
  a.K = pg->K;
  a.mass = mass->mass;
  a.born = mass->born;
  a.total = mass->total;
  a.N = N;
  a.M = M;
  a.Hq = Hq;
  a.H = pg->H;
  a.g = Hq / pg->H;
  a.B = pg->B;
  a.max_pages = pg->max_pages;
  while ((1 << a.page_shift) < pg->page) ++a.page_shift;
  a.n_pages = pg->n_pages;
  a.block = block;
  a.scale = scale;
  a.decay = decay;
  a.part = (float*)ws;
  a.G = kCtas;
  a.split = mass_split(a, kTQ);
  a.rows_lo = 0;
  a.rows_hi = 0x7fffffff;
  // Branches of a few rows (single tokens) and of many each have their kernel.  The
  // lengths are not known here: where only one kind is to be expected, its kernel
  // takes all (a launch for nothing costs 3 us; each kernel is right for any number).
  // M counts rows of padding too: 16 single tokens in a call for 6,240 go to the kernel
  // for many rows (40 heads over 4,681 keys 229 us, 115 us in a call for 16; 12 heads in
  // 32 bits 202 and 68 us).
  const bool bf16 = pg->dt == FASTAR_BF16;
  const int D = pg->D, limit = bf16 ? kMassFew : kMassFew32;
  const long long tall = (long long)M * a.g;
  // (The tensor cores' kernel holds lse / scale in 32 bits, which is a number there for
  // |lse| < 3e8 as long as the scale is not below 1e-30, and is cut below 2^-126 for
  // scales above 1e30; the kernel for a few rows needs no such quotient.)
  const bool fair = !bf16 || (scale >= 1e-30f && scale <= 1e30f);
  const bool many = fair && tall > 2ll * limit + 4ll * pg->B, few = !many || tall <= (bf16 ? 2ll : 1ll) * limit * pg->B;
  int rc = FASTAR_OK;
  if (few) {
    if (many) a.rows_hi = limit;
    rc = launch_mass_few(D, bf16, a, st, s);
    a.rows_lo = limit;
    a.rows_hi = 0x7fffffff;
  }
  if (rc != FASTAR_OK || !many) return rc;
  if (bf16) return launch_mass_tc(D, a, st, s);
  return D == 128 ? launch_t<128>(a, st, s) : launch_t<64>(a, st, s);
}

}  // namespace fastar
