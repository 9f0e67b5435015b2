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

// Checks the lengths and writes the prefix sums of the units: one CTA, a lane
// per branch; the row tiles of a branch behind its first kOwnTiles are counted
// by its whole warp.  Bound by the latency of a few rounds of loads and
// atomics (512 branches: about 15 us).
constexpr int kOwnTiles = 4;

__global__ void __launch_bounds__(kPlanThreads) branch_plan_kernel(BranchArgs a, int32_t* st) {
  pdl_wait();
  __shared__ long long sh[33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // nothing to do for the kernels behind: their loaders read the lists before
  // they know of the status, so these are written in any case, and also where
  // the call has no status word
  auto no_units = [&]() {
    for (int h = tid; h <= a.H + 1; h += kPlanThreads) a.head[h] = 0;
  };
  if (block_status_bad(st)) {
    no_units();
    return;
  }
  for (int t = tid; t <= a.ntiles; t += kPlanThreads) a.tile[t] = 0;
  __syncthreads();
  bool bad = false;
  auto add = [&](int t, int lo, int hi, int len) {
    const int T1 = (int)((((long long)t + 1) * a.TM + a.g - 1) / a.g);
    const int keys = branch_limit(min(hi, T1) - 1 - lo, hi - lo, len, a.block);
    atomicAdd((unsigned long long*)&a.tile[t], (unsigned long long)key_units(keys, a.TN));
  };
  for (int b0 = warp * 32; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + lane;
    int lo = 0, hi = 0, len = 0;
    if (b < a.B) {
      lo = a.cu[b];
      hi = a.cu[b + 1];
      len = a.len[b];
      if (!branch_ok(a, b, lo, hi, len)) {
        bad = true;
        hi = lo = 0;
      }
    }
    const int t0 = lo * a.g / a.TM, t1 = hi > lo ? (hi * a.g - 1) / a.TM : t0 - 1;
    for (int t = t0; t <= min(t1, t0 + kOwnTiles - 1); ++t) add(t, lo, hi, len);
    for (unsigned more = __ballot_sync(0xffffffffu, t1 >= t0 + kOwnTiles); more; more &= more - 1) {
      const int src = __ffs(more) - 1;
      const int l = __shfl_sync(0xffffffffu, lo, src), r = __shfl_sync(0xffffffffu, hi, src);
      const int n = __shfl_sync(0xffffffffu, len, src);
      const int last = __shfl_sync(0xffffffffu, t1, src);
      for (int t = __shfl_sync(0xffffffffu, t0, src) + kOwnTiles + lane; t <= last; t += 32) add(t, l, r, n);
    }
  }
  for (int h = tid; h < a.H; h += kPlanThreads)
    if (a.size && (a.size[h] < 0 || a.size[h] > a.C)) bad = true;
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (__syncthreads_or(bad)) {
    no_units();
    return;
  }
  const long long rows = (long long)a.cu[a.B] * a.g;
  const int nt = (int)((rows + a.TM - 1) / a.TM);
  long long carry = 0, total;
  for (int t0 = 0; t0 < nt; t0 += kPlanThreads) {
    const int t = t0 + tid;
    // (summed in L2; an item over nothing still has a unit, to be written)
    const long long v = t < nt ? max(1ll, __ldcg(&a.tile[t])) : 0;
    const long long x = block_scan_ll(v, sh, &total);
    if (t < nt) a.tile[t] = carry + x;
    carry += total;
  }
  if (tid == 0) a.tile[nt] = carry;
  const long long pages = carry;
  carry = 0;
  for (int h0 = 0; h0 < a.H; h0 += kPlanThreads) {
    const int h = h0 + tid;
    const long long v = h < a.H ? (long long)nt * (key_units(prefix_size(a, h), a.TN) + a.item_units) + pages : 0;
    const long long x = block_scan_ll(v, sh, &total);
    if (h < a.H) a.head[h] = carry + x;
    carry += total;
  }
  // (bad is false here) more than the walk's integers hold?
  for (int t = tid; t < nt; t += kPlanThreads) bad = bad || a.tile[t + 1] - a.tile[t] > kMaxUnits;
  bad = __syncthreads_or(bad || carry > (long long)kMaxUnits * a.G) != 0;
  if (tid == 0) {
    if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
    a.head[a.H] = nt > 0 && !bad ? carry : 0;
    a.head[a.H + 1] = nt;
  }
  pdl_trigger();
}

// Joins the partials of every item that is cut: grid (records, row groups); the
// run that begins an item left a record of it.  A warp takes 8 rows by 16
// columns: lane = row + 8 sub, and sub-group `sub` adds the partials of every
// fourth run, so that a few rows over many runs still keep four loads of each
// lane in flight; the four sums are joined by shuffles (a fixed order).  Bound
// by the latency of its launch and three round trips: 3.5 us of a short call.
constexpr int kJoinThreads = 256;

// kAhead: partials of a lane in one round trip.
template <typename T, int kAhead>
__global__ void __launch_bounds__(kJoinThreads) branch_combine_kernel(BranchArgs a, int32_t* st) {
  branch_touch(a, st);
  pdl_wait();
  const bool stop = status_bad(st);
  const BranchCut x = a.cuts[blockIdx.x];
  const int rows = a.cu[a.B] * a.g;
  // an item of padding alone has no record
  if (stop || (a.by_item && (int)(blockIdx.x % a.ntiles) * a.TM >= rows) || x.h < 0) return;
  // nor has one whose run gave up a wait, which a call without a status word
  // does not see: nothing out of range is followed
  if (x.h >= a.H || x.t < 0 || x.t >= a.ntiles || x.run < 0 || x.last < x.run || x.last >= a.G || x.slot >> 1 != x.run ||
      x.parts < 0 || x.parts > a.G)
    return;
  const int lane = threadIdx.x & 31, c = x.run;
  const int w = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5), groups = a.D / 16;
  const int i = w / groups * 8 + (lane & 7), col = w % groups * 16, sub = lane >> 3;
  const int r0 = x.t * a.TM;
  const int nr = min(a.TM, rows - r0), n = x.last - c + 1;
  if (w / groups * 8 >= nr) return;
  const bool live = i < nr;
  // the slot of the item's k-th run, -1 where that run is empty
  auto slot_of = [&](int k) {
    const int j = c + k;
    if (x.empty(a, j)) return -1;
    return j == c ? x.slot : 2 * j;
  };
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  for (int k0 = sub; k0 < n; k0 += 4 * kAhead) {
    // kAhead partials at a time, their statistics and columns in one round trip
    float2 ml[kAhead];
    float4 p[kAhead][4];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = k0 + 4 * q, slot = live && k < n ? slot_of(k) : -1;
      ml[q] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[q][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slot >= 0) {
        ml[q] = a.pml[(size_t)slot * a.slot_rows + i];
        const float4* po =
            reinterpret_cast<const float4*>(a.po + (size_t)slot * a.slot_rows * a.D) + (size_t)(col / 4) * a.slot_rows + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[q][e] = po[(size_t)e * a.slot_rows];
      }
    }
    float mn = m;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) mn = fmaxf(mn, ml[q].y != 0.f ? ml[q].x : -INFINITY);
    const float nb = mn == -INFINITY ? 0.f : mn, alpha = l == 0.f ? 0.f : exp2f(m - nb);
    l *= alpha;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] *= alpha;
    m = mn;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (ml[q].y == 0.f) continue;  // the row saw nothing in that run
      const float w = exp2f(ml[q].x - nb);
      l += w * ml[q].y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[4 * e] = fmaf(w, p[q][e].x, o[4 * e]);
        o[4 * e + 1] = fmaf(w, p[q][e].y, o[4 * e + 1]);
        o[4 * e + 2] = fmaf(w, p[q][e].z, o[4 * e + 2]);
        o[4 * e + 3] = fmaf(w, p[q][e].w, o[4 * e + 3]);
      }
    }
  }
  // the four sub-groups on one maximum
  float top = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
  const float base = top == -INFINITY ? 0.f : top, scale = l == 0.f ? 0.f : exp2f(m - base);
  l *= scale;
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] *= scale;
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    o[e] += __shfl_xor_sync(0xffffffffu, o[e], 8);
    o[e] += __shfl_xor_sync(0xffffffffu, o[e], 16);
  }
  if (live && sub == 0) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] *= inv;
    const int row = r0 + i;
    const size_t at = (size_t)(x.h * a.g + row % a.g) * a.N + row / a.g;
    T* out = (T*)a.out + at * a.D + col;
    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
    for (int e = 0; e < 16; e += V) st_vec<T, V>(out + e, o + e);
    if (a.lse && col == 0) a.lse[at] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
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
  const int warps = kJoinThreads / 32;
  const dim3 grid(a.by_item ? a.H * a.ntiles : a.G, ((rows + 7) / 8 * (a.D / 16) + warps - 1) / warps);
  // four where items have more than eight parts (4 tokens of 12 heads, 12 parts:
  // 17.4 us, 17.8 us by two), else two (64 tokens of 5 heads a group, about 7
  // parts: 111 us, 114 us by four, which leaves room for fewer CTAs)
  const bool many = a.by_item && a.G > 8 * a.H * a.ntiles;
  auto kernel = dt == FASTAR_BF16 ? (many ? branch_combine_kernel<__nv_bfloat16, 4> : branch_combine_kernel<__nv_bfloat16, 2>)
                                  : (many ? branch_combine_kernel<float, 4> : branch_combine_kernel<float, 2>);
  const cudaError_t rc = launch_pdl(kernel, grid, dim3(kJoinThreads), 0, s, a, st);
  if (rc != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "branch_combine");
  return FASTAR_OK;
}

namespace {
// Where items are not cut, a run's items count this many units each beside
// their own: their queries, first softmax and output (9 ragged prompts, 256
// items: 29.5 us; 31.4 us by units alone, 29.6 us at 6).
constexpr int kItemUnits = 3;
// Units, runs and partials of a call.  bf16: one CTA per SM, 256 (wide) or
// 128 rows and 128 keys; fp32: two CTAs per SM, 64 rows and 64 keys.
constexpr int kSms = 152;
struct Geometry {
  int TM, TN, G, ntiles, slot_rows;
  size_t cuts, head, tile, po, pml;  // bytes of the workspace's parts
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
Geometry geometry(fastar_dtype dt, bool wide, int H, long long rows, int D) {
  Geometry x;
  x.TM = dt == FASTAR_F32 ? 64 : wide ? 256 : 128;
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
  for (int k = 0; k < 3; ++k) {
    const Geometry x = geometry(k == 2 ? FASTAR_F32 : FASTAR_BF16, k == 1, H, (long long)N * (Hq / H), D);
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
  // 256 rows per item pay where most of the keys concern most of them and the
  // runs are long: every tile that is loaded then feeds four products.  So
  // where a branch fills them (two branches of 4680 tokens, 12 heads, 42,000
  // keys: 1.92 ms, 2.33 ms at 128 rows), or where the prefix is longer than
  // the pages of all branches of an item together and few rows are padding
  // (512 single tokens of 5 heads a group over 32,768 + 256 keys: 414 us, 473
  // us).  Otherwise most of a wide item idles while its pages pass (64 of those
  // tokens, up to 2048 keys of their own: 137 us, 111 us at 128 rows), and short
  // runs are latency alone (9 ragged prompts of up to 858 keys: 36.5 us, 29.6
  // us).  Tables, prefix and N have room for as much; the lengths are not known
  // here.
  const long long rows = (long long)N * a.g;
  const long long own = (long long)a.max_pages << a.page_shift, keys = a.C + own;
  const long long wide_tiles = (rows + 255) / 256, narrow_tiles = (rows + 127) / 128;
  const bool shared =
      8 * wide_tiles <= 5 * narrow_tiles && key_units(a.C, 128) * rows >= 256ll * a.B * ((own + 127) / 128);
  const bool wide = (rows / a.B >= 256 || shared) && a.H * wide_tiles * ((keys + 127) / 128) >= 16 * kSms;
  const Geometry x = geometry(dt, wide, a.H, rows, a.D);
  a.TM = x.TM;
  a.TN = x.TN;
  a.G = x.G;
  a.ntiles = x.ntiles;
  a.slot_rows = x.slot_rows;
  const long long units = key_units(a.C, a.TN) + a.B * (((long long)a.max_pages << a.page_shift) / a.TN + 1);
  a.planned = a.ntiles > kMaxTiles || (a.ntiles > kFewTiles && a.B > kMaxBranches) || units > kFewUnits / a.ntiles;
  const long long items = (long long)a.H * a.ntiles;
  a.whole = branch_whole(items, a.G, a.TM, a.TN, rows, a.B, a.C, own);
  a.item_units = a.whole ? kItemUnits : 0;
  a.by_item = items <= a.G;
  char* w = (char*)ws;
  a.cuts = (BranchCut*)w;
  a.head = (long long*)(w += x.cuts);
  a.tile = (long long*)(w += x.head);
  a.po = (float*)(w += x.tile);
  a.pml = (float2*)(w + x.po);
  int rc = a.planned ? launch_branch_plan(a, st, s) : FASTAR_OK;
  if (rc == FASTAR_OK) rc = dt == FASTAR_BF16 ? launch_branch_tc(a, st, s) : launch_branch_simt(a, st, s);
  if (rc == FASTAR_OK && !a.whole) rc = launch_branch_combine(a, dt, st, s);
  return rc;
}

}  // namespace fastar
