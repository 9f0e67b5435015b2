// Schedule shared by the kernels of fastar_branch_attention.
//
// For key/value head h the queries of its group form one matrix of N g rows,
// row r = token r / g, head h g + r % g: a row tile holds consecutive tokens,
// so consecutive branches.  The keys of a row tile are the live prefix rows,
// read once for every branch of the tile, followed by the page keys of each
// branch that has tokens in the tile.  A unit is TN of those keys.  All units
// of all (head, row tile) items are laid end to end, head after head, and cut
// into G equal runs, one per CTA: the split along a long cache needs no
// special case, no CTA waits for a longer one, and the cut depends on the
// lengths alone, so results do not change from run to run.  An item inside
// one run is finished there; one that is cut leaves a partial (O in fp32,
// running max and sum) per run, and branch_combine joins them in order.
//
// The lengths live on the device, so branch_plan computes the prefix sums of
// the units there; every consumer finds its place in them by searching.
#pragma once

#include "common.cuh"

namespace fastar {

struct BranchArgs {
  const void* q;
  const int32_t* cu;      // [B + 1]
  const int32_t* len;     // [B]
  const int32_t* table;   // [B][max_pages]
  const void* pK;         // [H][C][D] prefix
  const void* pV;
  const int32_t* m;       // [H][C] or null
  const int32_t* size;    // [H] or null (C)
  const void* K;          // pages
  const void* V;
  int N, Hq, H, g, B, C, D, max_pages, page_shift, n_pages, block;
  float scale;
  void* out;
  float* lse;
  // schedule
  int TM, TN, G, ntiles;  // ntiles: row tiles of all N tokens
  int slot_rows;          // rows of a partial
  long long* head;        // [H + 1] first unit of each head; then [2] rows in use, tiles in use
  long long* tile;        // [ntiles + 1] first page unit of each row tile
  float* po;              // [2 G][slot_rows][D]
  float2* pml;            // [2 G][slot_rows]
};

// Keys of its branch that token i of n (branch length len) sees.
__device__ __forceinline__ int branch_limit(int i, int n, int len, int block) {
  if (block <= 0) return len;
  const int t = len - n + i;
  if (t < 0) return 0;
  const int blocks = t / block + 1;
  return blocks > len / block ? len : blocks * block;
}
__device__ __forceinline__ int prefix_size(const BranchArgs& a, int h) {
  return a.size ? min(max(a.size[h], 0), a.C) : a.C;
}
__device__ __forceinline__ int prefix_units(int size, int TN) { return max(1, (size + TN - 1) / TN); }

// Entries of the ascending list x[0..n) that are <= v (whole warp).
template <typename T>
__device__ __forceinline__ int warp_count_le(const T* x, int n, T v) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // every entry below lo is <= v, none from hi on is
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < hi && x[at] <= v);
    const int k = __popc(m);  // probes <= v are the first k
    if (k == 0) return lo;
    const int nlo = lo + (k - 1) * step + 1;
    hi = min(hi, lo + k * step);
    lo = nlo;
  }
  const unsigned m = __ballot_sync(0xffffffffu, lo + lane < hi && x[lo + lane] <= v);
  return lo + __popc(m);
}

// One unit of work, as the consumers see it.
struct BranchUnit {
  int h, t;        // item
  int k0, nk;      // keys k0 .. k0 + nk - 1 (prefix rows or branch positions)
  int branch;      // -1: prefix
  int lo, n, len;  // the branch's first token, tokens and length
  int flags;       // 1 first unit of the item in this run, 2 last, 4 the run holds the whole item
  int slot;        // partial slot of the item
};

// Walks the units of CTA run c, a whole warp in step.
struct BranchWalk {
  long long u, u_end, istart, iend, run0;
  int h, t, c, nt, P, size;
  int T0, T1;
  // 32 branches at a time, one per lane: its tokens, length, visible keys and
  // the units up to and with it
  int bbase, before, total, lo, n, len, keys, nu, incl;

  __device__ __forceinline__ void load_batch(const BranchArgs& a) {
    const int b = bbase + (threadIdx.x & 31);
    lo = n = len = keys = nu = 0;
    if (b < a.B) {
      lo = a.cu[b];
      const int hi = a.cu[b + 1];
      n = hi - lo;
      len = a.len[b];
      const int last = min(hi, T1) - 1;
      if (last >= max(lo, T0)) keys = branch_limit(last - lo, n, len, a.block);
      nu = (keys + a.TN - 1) / a.TN;
    }
    incl = warp_incl_scan(nu);
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  __device__ __forceinline__ void enter(const BranchArgs& a) {
    const int rows = (int)a.head[a.H + 1];
    const int r0 = t * a.TM, r1 = min(r0 + a.TM, rows);
    T0 = r0 / a.g;
    T1 = (r1 + a.g - 1) / a.g;
    const int hs = prefix_size(a, h);
    size = hs;
    P = prefix_units(hs, a.TN);
    iend = istart + P + (a.tile[t + 1] - a.tile[t]);
    // first branch with tokens at or behind T0 (empty ones contribute nothing)
    bbase = max(0, warp_count_le(a.cu, a.B, T0) - 1);
    before = 0;
    load_batch(a);
  }
  // false: nothing to do for this CTA
  __device__ __forceinline__ bool start(const BranchArgs& a, int cta) {
    c = cta;
    const long long U = a.head[a.H];
    nt = (int)a.head[a.H + 2];
    u = run0 = U * c / a.G;
    u_end = U * (c + 1) / a.G;
    if (u >= u_end) return false;
    h = warp_count_le(a.head, a.H, u) - 1;
    const long long off = u - a.head[h];
    const int p = prefix_units(prefix_size(a, h), a.TN);
    // the row tile t with t p + tile[t] <= off < (t + 1) p + tile[t + 1]
    const int lane = threadIdx.x & 31;
    int l = 0, r = nt;
    while (r - l > 1) {
      const int step = (r - l + 31) / 32;
      const int at = l + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, at < r && (long long)at * p + a.tile[at] <= off);
      const int k = max(1, __popc(m));
      r = min(r, l + k * step);
      l = l + (k - 1) * step;
    }
    t = l;
    istart = a.head[h] + (long long)t * p + a.tile[t];
    enter(a);
    return true;
  }
  // The next unit; false at the end of the run.
  __device__ __forceinline__ bool next(const BranchArgs& a, BranchUnit& x) {
    if (u >= u_end) return false;
    if (u >= iend) {
      istart = iend;
      if (++t == nt) {
        t = 0;
        ++h;
      }
      enter(a);
    }
    const int off = (int)(u - istart);
    x.h = h;
    x.t = t;
    const bool whole = istart >= run0 && iend <= u_end;
    x.flags = ((u == istart || u == run0) ? 1 : 0) | ((u + 1 == iend || u + 1 == u_end) ? 2 : 0) | (whole ? 4 : 0);
    x.slot = 2 * c + (istart <= run0 ? 0 : 1);
    if (off < P) {
      x.branch = -1;
      x.k0 = off * a.TN;
      x.nk = max(0, min(a.TN, size - x.k0));
      x.lo = x.n = x.len = 0;
    } else {
      int s = off - P - before;
      while (s >= total && bbase < a.B) {
        before += total;
        s -= total;
        bbase += 32;
        load_batch(a);
      }
      const unsigned m = __ballot_sync(0xffffffffu, incl > s);
      const int src = m ? __ffs(m) - 1 : 31;
      const int k = s - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, nu, src));
      x.branch = bbase + src;
      x.lo = __shfl_sync(0xffffffffu, lo, src);
      x.n = __shfl_sync(0xffffffffu, n, src);
      x.len = __shfl_sync(0xffffffffu, len, src);
      x.k0 = k * a.TN;
      x.nk = max(0, min(a.TN, __shfl_sync(0xffffffffu, keys, src) - x.k0));
    }
    ++u;
    return true;
  }
};

// Keys of unit x (counted from x.k0) that row r of its item sees.
__device__ __forceinline__ int branch_row_keys(const BranchArgs& a, const BranchUnit& x, int r) {
  if (x.branch < 0) return x.nk;
  const int i = r / a.g - x.lo;
  if (i < 0 || i >= x.n) return 0;
  return max(0, min(x.nk, branch_limit(i, x.n, x.len, a.block) - x.k0));
}

int launch_branch_plan(const BranchArgs& a, int32_t* st, cudaStream_t s);
int launch_branch_combine(const BranchArgs& a, fastar_dtype dt, int32_t* st, cudaStream_t s);
int launch_branch_simt(const BranchArgs& a, int32_t* st, cudaStream_t s);
int launch_branch_tc(const BranchArgs& a, int32_t* st, cudaStream_t s);

}  // namespace fastar
