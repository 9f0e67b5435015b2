// fastar_branch_attention: the plan of its units, the join of its partials,
// workspace layout and dispatch.
#include <math.h>

#include "branch.cuh"

namespace fastar {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long block_scan_ll(long long v, long long* sh, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    long long w = sh[lane], wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += x;
    }
    sh[lane] = wi - w;
    if (lane == 31) sh[32] = wi;
  }
  __syncthreads();
  const long long res = sh[warp] + inc - v;
  *total = sh[32];
  __syncthreads();
  return res;
}

// Checks the lengths and writes the prefix sums of the units: one CTA, a warp
// per branch and a lane per row tile that the branch touches.
__global__ void __launch_bounds__(kPlanThreads) branch_plan_kernel(BranchArgs a, int32_t* st) {
  pdl_wait();
  __shared__ long long sh[33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (block_status_bad(st)) return;
  for (int t = tid; t <= a.ntiles; t += kPlanThreads) a.tile[t] = 0;
  __syncthreads();
  bool bad = false;
  for (int b = warp; b < a.B; b += kPlanThreads / 32) {
    const int lo = a.cu[b], hi = a.cu[b + 1], len = a.len[b];
    if (!branch_ok(a, b, lo, hi, len)) {
      bad = true;
      continue;
    }
    if (hi == lo) continue;
    const int t0 = (int)((long long)lo * a.g / a.TM), t1 = (int)(((long long)hi * a.g - 1) / a.TM);
    for (int t = t0 + lane; t <= t1; t += 32) {
      const int T1 = (int)((((long long)t + 1) * a.TM + a.g - 1) / a.g);
      const int keys = branch_limit(min(hi, T1) - 1 - lo, hi - lo, len, a.block);
      atomicAdd((unsigned long long*)&a.tile[t], (unsigned long long)((keys + a.TN - 1) / a.TN));
    }
  }
  for (int h = tid; h < a.H; h += kPlanThreads)
    if (a.size && (a.size[h] < 0 || a.size[h] > a.C)) bad = true;
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (__syncthreads_or(bad)) {
    // nothing to do for the kernels behind, also without a status word
    for (int h = tid; h <= a.H + 1; h += kPlanThreads) a.head[h] = 0;
    return;
  }
  const long long rows = (long long)a.cu[a.B] * a.g;
  const int nt = (int)((rows + a.TM - 1) / a.TM);
  long long carry = 0, total;
  for (int t0 = 0; t0 < nt; t0 += kPlanThreads) {
    const int t = t0 + tid;
    const long long v = t < nt ? __ldcg(&a.tile[t]) : 0;  // summed in L2
    const long long x = block_scan_ll(v, sh, &total);
    if (t < nt) a.tile[t] = carry + x;
    carry += total;
  }
  if (tid == 0) a.tile[nt] = carry;
  const long long pages = carry;
  carry = 0;
  for (int h0 = 0; h0 < a.H; h0 += kPlanThreads) {
    const int h = h0 + tid;
    const long long v = h < a.H ? (long long)nt * prefix_units(prefix_size(a, h), a.TN) + pages : 0;
    const long long x = block_scan_ll(v, sh, &total);
    if (h < a.H) a.head[h] = carry + x;
    carry += total;
  }
  if (tid == 0) {
    a.head[a.H] = nt > 0 ? carry : 0;
    a.head[a.H + 1] = nt;
  }
  pdl_trigger();
}

// Joins the partials of every item that is cut: grid (runs, row groups), a
// warp per row; the run that begins an item left a record of it.  The
// maxima and sums of up to 32 partials are read at once, one per lane, then
// the rows of O eight at a time, in the order of the runs.
constexpr int kJoinRows = 16;  // rows per CTA, two per warp

template <typename T>
__global__ void __launch_bounds__(256) branch_combine_kernel(BranchArgs a, int32_t* st) {
  pdl_wait();
  const bool stop = status_bad(st);
  const BranchCut x = a.cuts[blockIdx.x];
  if (stop || x.h < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  const int rows = a.cu[a.B] * a.g, r0 = x.t * a.TM;
  const int nr = min(a.TM, rows - r0), n = x.last - c + 1;
  for (int i = blockIdx.y * kJoinRows + warp; i < min(nr, (int)(blockIdx.y + 1) * kJoinRows); i += 8) {
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += 32) {
      // run c + j0 + lane: its slot, or none where it is past the item or empty
      const int j = c + j0 + lane;
      int slot = j == c ? x.slot : 2 * j;
      if (j0 + lane >= n || x.U * j / a.G == x.U * (j + 1) / a.G) slot = -1;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (slot >= 0) ml = a.pml[(size_t)slot * a.slot_rows + i];
      if (ml.y == 0.f) slot = -1;  // the row saw nothing in that run
      float top = slot >= 0 ? ml.x : -INFINITY;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
      const float w = slot >= 0 ? exp2f(ml.x - base) : 0.f;
      const float alpha = l == 0.f ? 0.f : exp2f(m - base);
      l = l * alpha + warp_sum(slot >= 0 ? w * ml.y : 0.f);
      m = mn;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= alpha;
      for (int k0 = 0; k0 < min(32, n - j0); k0 += 8) {
        float4 p[8];
        float wk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int sk = __shfl_sync(0xffffffffu, slot, k0 + k);
          wk[k] = __shfl_sync(0xffffffffu, w, k0 + k);
          p[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (sk >= 0 && lane * 4 < a.D)
            p[k] = *reinterpret_cast<const float4*>(a.po + ((size_t)sk * a.slot_rows + i) * a.D + lane * 4);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[0] = fmaf(wk[k], p[k].x, o[0]);
          o[1] = fmaf(wk[k], p[k].y, o[1]);
          o[2] = fmaf(wk[k], p[k].z, o[2]);
          o[3] = fmaf(wk[k], p[k].w, o[3]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= inv;
    const int row = r0 + i;
    const size_t at = (size_t)(x.h * a.g + row % a.g) * a.N + row / a.g;
    if (lane * 4 < a.D) st_vec<T, 4>((T*)a.out + at * a.D + lane * 4, o);
    if (a.lse && lane == 0)
      a.lse[at] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.6931471805599453f;
  }
  pdl_trigger();
}

}  // namespace

int launch_branch_plan(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  if (launch_pdl(branch_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "branch_plan");
  return FASTAR_OK;
}

int launch_branch_combine(const BranchArgs& a, fastar_dtype dt, int32_t* st, cudaStream_t s) {
  const int rows = (int)min((long long)a.TM, (long long)a.N * a.g);
  const dim3 grid(a.G, (rows + kJoinRows - 1) / kJoinRows);
  cudaError_t rc = dt == FASTAR_BF16 ? launch_pdl(branch_combine_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a, st)
                                     : launch_pdl(branch_combine_kernel<float>, grid, dim3(256), 0, s, a, st);
  if (rc != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "branch_combine");
  return FASTAR_OK;
}

namespace {
// Units, runs and partials of a call.  bf16: one CTA per SM, 256 rows and 128
// keys (128 rows where that is all there is); fp32: two CTAs per SM, 64 rows
// and 64 keys.
constexpr int kSms = 152;
struct Geometry {
  int TM, TN, G, ntiles, slot_rows;
  size_t cuts, head, tile, po, pml;  // bytes of the workspace's parts
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
Geometry geometry(fastar_dtype dt, int H, long long rows, int D) {
  Geometry x;
  x.TM = dt == FASTAR_F32 ? 64 : rows <= 128 ? 128 : 256;
  x.TN = dt == FASTAR_F32 ? 64 : 128;
  x.G = dt == FASTAR_F32 ? 2 * kSms : kSms;
  x.ntiles = (int)((rows + x.TM - 1) / x.TM);
  x.slot_rows = (int)(rows < x.TM ? rows : x.TM);
  x.cuts = up256((size_t)x.G * sizeof(BranchCut));
  x.head = up256((size_t)(H + 2) * 8);
  x.tile = up256((size_t)(x.ntiles + 1) * 8);
  x.po = up256((size_t)2 * x.G * x.slot_rows * D * 4);
  x.pml = up256((size_t)2 * x.G * x.slot_rows * 8);
  return x;
}
}  // namespace

size_t branch_ws_bytes(int Hq, int H, int N, int D) {
  if (Hq < 1 || H < 1 || N < 1 || D < 1 || Hq % H) return 0;
  size_t most = 0;
  for (fastar_dtype dt : {FASTAR_BF16, FASTAR_F32}) {
    const Geometry x = geometry(dt, H, (long long)N * (Hq / H), D);
    const size_t n = x.cuts + x.head + x.tile + x.po + x.pml;
    if (n > most) most = n;
  }
  return most;
}

int launch_branch(fastar_dtype dt, const void* q, int Hq, int N, const int32_t* cu, const fastar_prefix* px,
                  const fastar_pages* pg, float scale, int block, void* out, float* lse, void* ws, int32_t* st,
                  cudaStream_t s) {
  BranchArgs a = {};
  a.q = q;
  a.cu = cu;
  a.len = pg->len;
  a.table = pg->table;
  a.K = pg->K;
  a.V = pg->V;
  if (px) {
    a.pK = px->K;
    a.pV = px->V;
    a.m = px->m;
    a.size = px->size;
    a.C = px->C;
  }
  a.N = N;
  a.Hq = Hq;
  a.H = pg->H;
  a.g = Hq / pg->H;
  a.B = pg->B;
  a.D = pg->D;
  a.max_pages = pg->max_pages;
  a.n_pages = pg->n_pages;
  while ((1 << a.page_shift) < pg->page) ++a.page_shift;
  a.block = block;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  const Geometry x = geometry(dt, a.H, (long long)N * a.g, a.D);
  a.TM = x.TM;
  a.TN = x.TN;
  a.G = x.G;
  a.ntiles = x.ntiles;
  a.slot_rows = x.slot_rows;
  char* w = (char*)ws;
  a.cuts = (BranchCut*)w;
  a.head = (long long*)(w += x.cuts);
  a.tile = (long long*)(w += x.head);
  a.po = (float*)(w += x.tile);
  a.pml = (float2*)(w + x.po);
  int rc = a.ntiles > 1 ? launch_branch_plan(a, st, s) : FASTAR_OK;
  if (rc == FASTAR_OK) rc = dt == FASTAR_BF16 ? launch_branch_tc(a, st, s) : launch_branch_simt(a, st, s);
  if (rc == FASTAR_OK) rc = launch_branch_combine(a, dt, st, s);
  return rc;
}

}  // namespace fastar
