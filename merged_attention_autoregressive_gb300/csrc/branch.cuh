// Schedule shared by the kernels of fastar_branch_attention.
//
// For key/value head h the queries of its group form one matrix of N g rows,
// row r = token r / g, head h g + r % g: a row tile holds consecutive tokens,
// so consecutive branches.  The keys of a row tile are the live prefix rows,
// read once for every branch of the tile, followed by the page keys of each
// branch that has tokens in the tile.  A unit is TN of those keys.  The units of
// all (head, row tile) items are laid end to end, head after head, and shared
// out to G runs, one per CTA, in one of three ways:
//   even   G equal runs, wherever they begin and end: the split along a long
//          cache needs no special case, and no CTA waits for a longer one;
//   parts  one row tile (single tokens): each head's item in the same number of
//          equal parts, so that no run has two items (branch_parts);
//   whole  many short items: a run ends where an item begins (branch_whole).
// The cut depends on the lengths alone, so results do not change from run to
// run.  An item inside one run is finished there; one that is cut leaves a
// partial (O in fp32, running max and sum) per run, and branch_combine joins them
// in order.
//
// The lengths live on the device.  Up to 8 row tiles, or 64 with at most 32
// branches, every CTA sums the units itself; with more, or where tables and
// prefix have room for more units than its integers hold (kFewUnits),
// branch_plan writes the prefix sums of the units first and each CTA finds its
// place in them by searching.
#pragma once

#include <math.h>

#include "common.cuh"

namespace fastar {

struct BranchCut;

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
  int planned;            // branch_plan has written head and tile
  int whole;              // items are not cut: a run ends where an item begins
  int item_units;         // whole: an item counts as so many units more
  int by_item;            // cuts has an entry per item (there are at most G), else per run
  BranchCut* cuts;        // [G] the items that are cut
  long long* head;        // planned: [H + 1] first unit of each head, then the tiles in use
  long long* tile;        // planned: [ntiles + 1] first page unit of each row tile
  float* po;              // [2 G][D / 4][slot_rows][4]: neighbouring rows lie side by side
  float2* pml;            // [2 G][slot_rows]
};

// Brings the call's arguments into the constant cache; before pdl_wait, so
// that their misses (one per 64 bytes) pass while the previous kernel ends.
__device__ __forceinline__ void branch_touch(const BranchArgs& a, const int32_t* st) {
  asm volatile("" ::"l"(a.q), "l"(a.size), "r"(a.N), "r"(a.max_pages), "l"(a.lse), "r"(a.G), "l"(a.head), "l"(a.pml),
               "l"(st));
}

// Keys of its branch that token i of n (branch length len) sees.
__device__ __forceinline__ int branch_limit(int i, int n, int len, int block) {
  if (block <= 0) return len;
  const int t = len - n + i;
  if (t < 0) return 0;
  const int blocks = t / block + 1;
  return blocks > len / block ? len : blocks * block;
}
// Units of TN keys that hold `keys` of them (up to 2^31 - 1, whose sum with TN
// is past an int).
__host__ __device__ __forceinline__ int key_units(int keys, int TN) {
  return (int)(((unsigned)keys + (unsigned)TN - 1) / (unsigned)TN);
}
__device__ __forceinline__ int prefix_size(const BranchArgs& a, int h) {
  return a.size ? min(max(a.size[h], 0), a.C) : a.C;
}

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

// Whether the lengths and offsets of a lane's branch hold.
__device__ __forceinline__ bool branch_ok(const BranchArgs& a, int b, int lo, int hi, int len) {
  return lo >= 0 && hi >= lo && hi <= a.N && (b != 0 || lo == 0) && len >= 0 &&
         (long long)len <= ((long long)a.max_pages << a.page_shift);
}

constexpr int kLaneTiles = 2;               // row tiles per lane of an unplanned call
constexpr int kMaxTiles = 32 * kLaneTiles;  // row tiles, and above kFewTiles of them
constexpr int kMaxBranches = 32;            // branches, of a call that goes without a plan
constexpr int kFewTiles = 8;
constexpr long long kFewUnits = 1 << 26;   // units of 32 heads fit an int: of a head without a plan
constexpr int kMaxUnits = 1 << 30;         // units of an item, and of a run

// First token of row tile t, and one behind its last.
__device__ __forceinline__ int tile_begin(const BranchArgs& a, int t) { return t * a.TM / a.g; }
__device__ __forceinline__ int tile_end(const BranchArgs& a, int t) { return ((t + 1) * a.TM + a.g - 1) / a.g; }

// What a run starts from (whole warp).  Few row tiles: summed from the
// lengths right here, so that single tokens and short prompts need no plan
// kernel; lane l holds tiles l and l + 32.  Otherwise from branch_plan's lists.
struct BranchPlace {
  long long U;            // units of the call; 0: nothing to do, or something does not hold
  int nt, sum;            // row tiles in use; page units of one head's tiles (unplanned)
  int pages[kLaneTiles];  // page units of the lane's tiles (unplanned)

  __device__ __forceinline__ void load(const BranchArgs& a, int32_t* st) {
    const int lane = threadIdx.x & 31;
    if (a.planned) {
      U = a.head[a.H];
      nt = (int)a.head[a.H + 1];
      return;
    }
    bool ok = true;
    sum = 0;
    const int size0 = a.size && lane < a.H ? a.size[lane] : a.C;  // on its way with the lengths
    int used = 0, t0[kLaneTiles], t1[kLaneTiles];
#pragma unroll
    for (int e = 0; e < kLaneTiles; ++e) {
      const int t = lane + 32 * e;
      pages[e] = 0;
      if (a.ntiles > kFewTiles) {
        t0[e] = t < a.ntiles ? tile_begin(a, t) : 0x7fffffff;
        t1[e] = t < a.ntiles ? tile_end(a, t) : 0;
      }
    }
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      int lo = 0, hi = 0, len = 0;
      if (b < a.B) {
        lo = a.cu[b];
        hi = a.cu[b + 1];
        len = a.len[b];
        ok = ok && branch_ok(a, b, lo, hi, len);
        if (!ok) hi = lo = 0;
      }
      used = max(used, hi);
      if (a.ntiles == 1) {
        if (hi > lo) sum += key_units(branch_limit(hi - 1 - lo, hi - lo, len, a.block), a.TN);
      } else if (a.ntiles <= kFewTiles) {
        // a branch per lane, the tiles one after the other
        for (int t = 0; t < a.ntiles; ++t) {
          const int last = min(hi, tile_end(a, t)) - 1;
          int v = 0;
          if (last >= max(lo, tile_begin(a, t))) v = key_units(branch_limit(last - lo, hi - lo, len, a.block), a.TN);
          v = __reduce_add_sync(0xffffffffu, v);
          if (lane == t) pages[0] += v;
        }
      } else {
        // a tile per lane, the branches one after the other
        for (int k = 0; k < min(32, a.B - b0); ++k) {
          const int l = __shfl_sync(0xffffffffu, lo, k), r = __shfl_sync(0xffffffffu, hi, k);
          const int n = __shfl_sync(0xffffffffu, len, k);
#pragma unroll
          for (int e = 0; e < kLaneTiles; ++e) {
            const int last = min(r, t1[e]) - 1;
            if (last >= max(l, t0[e])) pages[e] += key_units(branch_limit(last - l, r - l, n, a.block), a.TN);
          }
        }
      }
    }
    used = __reduce_max_sync(0xffffffffu, used);
    // an item over nothing still has a unit, to be written
    if (a.ntiles == 1) {
      nt = used > 0 ? 1 : 0;
      sum = max(1, __reduce_add_sync(0xffffffffu, sum));
    } else {
      nt = (used * a.g + a.TM - 1) / a.TM;
      sum = 0;
#pragma unroll
      for (int e = 0; e < kLaneTiles; ++e) {
        pages[e] = lane + 32 * e < nt ? max(1, pages[e]) : 0;
        sum += pages[e];
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
    }
    U = 0;
    for (int h0 = 0; h0 < a.H; h0 += 32) {
      const int h = h0 + lane;
      int v = 0;
      if (h < a.H) {
        const int size = h0 == 0 ? size0 : a.size ? a.size[h] : a.C;
        ok = ok && size >= 0 && size <= a.C;
        v = key_units(min(max(size, 0), a.C), a.TN) + a.item_units;
      }
      U += (long long)__reduce_add_sync(0xffffffffu, v) * nt + (long long)min(32, a.H - h0) * sum;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    if (!ok || nt == 0) U = 0;
  }
  // Units of the longest item of a call of one row tile (the sizes are in L1).
  __device__ __forceinline__ int longest_item(const BranchArgs& a) const {
    int v = 0;
#pragma unroll 1
    for (int h = threadIdx.x & 31; h < a.H; h += 32) v = max(v, prefix_size(a, h));
    return key_units(__reduce_max_sync(0xffffffffu, v), a.TN) + pages_of(a, 0);
  }
  // Page units of row tile t.
  __device__ __forceinline__ int pages_of(const BranchArgs& a, int t) const {
    if (a.planned) return (int)(a.tile[t + 1] - a.tile[t]);
    if (a.ntiles == 1) return sum;
    int v = 0;
#pragma unroll
    for (int e = 0; e < kLaneTiles; ++e) {
      const int x = __shfl_sync(0xffffffffu, pages[e], t & 31);
      if (t >> 5 == e) v = x;
    }
    return v;
  }
  // The item of unit u: head, row tile and first unit.
  __device__ __forceinline__ void find(const BranchArgs& a, long long u, int& h, int& t, long long& first) const {
    const int lane = threadIdx.x & 31;
    if (a.planned) {
      h = warp_count_le(a.head, a.H, u) - 1;
      const long long off = u - a.head[h];
      const int p = key_units(prefix_size(a, h), a.TN) + a.item_units;
      int l = 0, r = nt;  // the row tile t with t p + tile[t] <= off < (t + 1) p + tile[t + 1]
      while (r - l > 1) {
        const int step = (r - l + 31) / 32;
        const int at = l + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < r && (long long)at * p + a.tile[at] <= off);
        const int k = max(1, __popc(m));
        r = min(r, l + k * step);
        l = l + (k - 1) * step;
      }
      t = l;
      first = a.head[h] + (long long)t * p + a.tile[t];
      return;
    }
    h = t = 0;
    first = 0;
    int p = 0;
    for (int h0 = 0; h0 < a.H; h0 += 32) {
      const int x = h0 + lane;
      const int pu = x < a.H ? key_units(prefix_size(a, x), a.TN) + a.item_units : 0;
      const int v = x < a.H ? pu * nt + sum : 0;  // at most kFewUnits
      const int inc = warp_incl_scan(v);
      const unsigned m = __ballot_sync(0xffffffffu, x < a.H && first + inc > u);
      if (m) {
        const int src = __ffs(m) - 1;
        h = h0 + src;
        p = __shfl_sync(0xffffffffu, pu, src);
        first += __shfl_sync(0xffffffffu, inc - v, src);
        break;
      }
      first += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (nt == 1) return;
#pragma unroll
    for (int e = 0; e < kLaneTiles; ++e) {
      const int x = lane + 32 * e, v = x < nt ? p + pages[e] : 0;
      const int inc = warp_incl_scan(v);
      const unsigned m = __ballot_sync(0xffffffffu, x < nt && first + inc > u);
      if (m) {
        const int src = __ffs(m) - 1;
        t = 32 * e + src;
        first += __shfl_sync(0xffffffffu, inc - v, src);
        return;
      }
      first += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
};

// One unit of work, as the consumers see it.
struct BranchUnit {
  int h, t;        // item
  int k0, nk;      // keys k0 .. k0 + nk - 1 (prefix rows or branch positions)
  int branch;      // -1: prefix
  int lo, n, len;  // the branch's first token, tokens and length
  int flags;       // 1 first unit of the item in this run, 2 last, 4 the run holds the whole item
  int slot;        // partial slot of the item
};

// First unit of run c of G.
__device__ __forceinline__ long long branch_cut(long long U, int c, int G) {
  return U < (1 << 23) ? (long long)((unsigned)U * (unsigned)c / (unsigned)G) : U * c / G;
}

// What the join needs of an item that is cut.
struct BranchCut {
  int h, t;        // h = -1: none
  int run, last;   // the runs that begin and finish it
  int slot;        // the partial of the first; the later runs have slot 2 j
  int parts, len;  // the item's own equal parts of its len units; 0: cut with the rest
  long long U;

  // Whether run j has no unit.
  __device__ __forceinline__ bool empty(const BranchArgs& a, int j) const {
    if (parts) return part(len, j % parts, parts) == part(len, j % parts + 1, parts);
    return U < a.G && branch_cut(U, j, a.G) == branch_cut(U, j + 1, a.G);
  }
  // First unit of part p of n <= 304 of an item of len < 2^23 units.
  static __device__ __forceinline__ int part(int len, int p, int n) { return (unsigned)len * (unsigned)p / (unsigned)n; }
};

// Whether the items of a call are left whole: short items (a few microseconds
// each) are not cut where there are enough of them, since partials and join cost
// more than the imbalance (9 ragged prompts of up to 858 keys, 4 heads, 256
// items: 29.6 us, 37.3 us when cut; 40 prompts of 200 tokens over 300, 12 heads:
// 92 and 105 us; 300 of 20 over 300: 156 and 169 us).  rows: of all tokens of a
// head; B: branches; own: positions that a branch has room for.
//
// An item holds the keys of every branch with tokens in its row tile, `units` of
// them where the branches share the rows evenly.  Whole, some run takes one item
// more than others: that is weighed against the cut's cost (2,560 single tokens
// of 8 heads over 1,024 keys each, 160 items: 2.67 ms whole, 1.52 ms cut; fp32,
// whose units take 5 us: 16 prompts of 250 tokens, 8 heads 149 and 130 us).
// Branches of about one tile of rows on average are likely to be long ones beside
// short ones, and then a few tiles hold most of the keys (7 single tokens and a
// prompt of 1,024 tokens, 40 heads, causal: 126 us whole, 89 us cut).
constexpr int kWholeKeys = 8, kWholeUnits = 24;  // units of one branch, of an item
__host__ __device__ inline bool branch_whole(long long items, int G, int TM, int TN, long long rows, int B, int C,
                                             long long own) {
  if (items < G || (C + own + TN - 1) / TN > kWholeKeys) return false;
  const long long others = B * (long long)TM / rows;  // branches of a tile beside the first
  const long long units = key_units(C, TN) + (others + 1) * ((own + TN - 1) / TN);
  if (units > kWholeUnits || (others == 0 && 2 * rows < 3ll * TM * B)) return false;
  const long long cut = TN == 64 ? 2 : 12;  // partials and join, in units
  return (items + G - 1) / G * units * G <= items * units + cut * G;
}

// Parts of each of `items` items of U units together, the longest of `longest`,
// on G runs; 0: an even cut of all units instead.
//
// Few items: each in the same number of equal parts, when that makes a run at
// most kTwoItems units longer than an even cut of all units would.  An even cut
// gives some runs the end of an item and the begin of the next, and the queries,
// first softmax and output of two items cost that much more (4 branches of one
// token, 12 heads, 28 units each: 19.7 us, 17.4 us in parts).  The longest item
// decides: heads of a merged cache differ in their live rows (40 heads, one of
// 32,768 rows and the others of 1,200: 118 us in parts, 32 us by an even cut).
//
// A part more saves a share of the units' time and costs the join about 0.1 us:
// len / p units of 0.75 us (5 us on the FP32 pipes) and p of those are least near
// p = sqrt(8 len) (sqrt(48 len)).  One token of 2 heads, 23 units: 14.9 us in 14
// parts, 16.0 us in 17, 21.0 us in 76 (fp32, 45 units: 19.6 us in 47, 29.9 us in 17,
// 31.7 us in 152).
constexpr int kTwoItems = 4;
__host__ __device__ inline int branch_parts(long long U, int longest, int items, int G, bool fp32) {
  if (U >= (1 << 23)) return 0;
  const unsigned n = (unsigned)(G / items), u = (unsigned)U, g = (unsigned)G;
  if (((unsigned)longest + n - 1) / n > (u + g - 1) / g + kTwoItems) return 0;
  const int best = (int)ceilf(sqrtf((fp32 ? 48.f : 8.f) * (float)longest));
  return best < 1 ? 1 : best < (int)n ? best : (int)n;
}

// Walks the units of run c, a whole warp in step, a stretch of units of one
// branch (or of the prefix) at a time.
struct BranchWalk {
  BranchPlace place;
  int h, t, c, left;               // item; run; units left in the run
  int off, units, from;            // next unit of the item, its units, the first one in this run
  int P, size;                     // units and rows of the prefix
  int parts;                       // parts of each item; 0: an even cut of all units
  long long end;                   // even cut: end of the run
  int T0, T1;
  bool head_item;                  // the run's first item
  bool whole;
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
      nu = key_units(keys, a.TN);
    }
    incl = warp_incl_scan(nu);
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  __device__ __forceinline__ void enter(const BranchArgs& a, int at) {
    const int tokens = a.cu[a.B];
    T0 = a.ntiles > 1 ? tile_begin(a, t) : 0;
    T1 = a.ntiles > 1 ? min(tokens, tile_end(a, t)) : tokens;
    size = prefix_size(a, h);
    P = key_units(size, a.TN);
    units = P + place.pages_of(a, t);
    off = from = at;
    left -= a.item_units;
    whole = at == 0 && units <= left;

    // first branch with tokens at or behind T0 (empty ones contribute nothing)
    bbase = a.ntiles > 1 ? max(0, warp_count_le(a.cu, a.B, T0) - 1) : 0;
    before = 0;
    load_batch(a);
  }
  // Goes to the start of run cta; false: the run is empty.
  __device__ __forceinline__ bool start(const BranchArgs& a, int cta, int32_t* st) {
    place.load(a, st);
    c = cta;
    off = units = from = left = 0;
    head_item = true;
    const long long U = place.U;
    if (U == 0) {
      // no item: nothing for the join
      if (a.by_item && c == 0)
        for (int i = threadIdx.x & 31; i < a.H * a.ntiles; i += 32) a.cuts[i].h = -1;
      return false;
    }
    parts = 0;
    if (a.by_item && !a.whole && a.ntiles == 1) parts = branch_parts(U, place.longest_item(a), a.H, a.G, a.TM == 64);
    if (parts) {
      h = c / parts;
      t = 0;
      if (h >= a.H) return false;
      const int len = key_units(prefix_size(a, h), a.TN) + place.pages_of(a, t);
      const int u0 = BranchCut::part(len, c % parts, parts);
      left = BranchCut::part(len, c % parts + 1, parts) - u0;
      if (left > 0) enter(a, u0);
      return left > 0;
    }
    long long u = branch_cut(U, c, a.G), first = u;
    end = branch_cut(U, c + 1, a.G);
    if (a.whole && end < U) {
      place.find(a, end, h, t, first);
      end = first;
    }
    if (u < U) place.find(a, u, h, t, first);
    if (a.whole) u = u < U ? first : U;
    left = (int)(end - u);
    if (left > 0) enter(a, (int)(u - first));
    return left > 0;
  }
  // Writes the join's record of the present item, which the run has begun
  // (calls of few items; any time while the walk is there), or of the run.
  __device__ __forceinline__ void record(const BranchArgs& a, bool run) const {
    if (run == (a.by_item != 0) || (threadIdx.x & 31) || (!run && from != 0)) return;
    a.cuts[run ? c : h * a.ntiles + t] = cut(a);
  }
  // The join's record of the present item: a run that begins an item and does
  // not finish it names the run that does.
  __device__ __forceinline__ BranchCut cut(const BranchArgs& a) const {
    BranchCut x = {-1, 0, 0, 0, 0, parts, units, place.U};
    if (from == 0 && units - off > left) {
      x.h = h;
      x.t = t;
      x.run = c;
      x.slot = 2 * c + (head_item ? 0 : 1);
      const long long last = end - left - off + units, U = place.U;  // one behind the item's last unit
      x.last = parts ? c / parts * parts + parts - 1 : U < (1 << 23) ? (int)(((unsigned)last * (unsigned)a.G - 1) / (unsigned)U) : (int)((last * a.G - 1) / U);
    }
    return x;
  }
  // The next stretch: x describes its first unit, `count` units follow one
  // another, `keys_end` bounds their keys.  False at the end of the run.
  // first / last: whether the stretch opens / closes the item in this run.
  __device__ __forceinline__ bool next(const BranchArgs& a, BranchUnit& x, int& count, int& keys_end, bool& opens,
                                       bool& closes, int opened) {
    if (left == 0) return false;
    if (off == units) {
      if (++t == place.nt) {
        t = 0;
        ++h;
      }
      head_item = false;
      enter(a, 0);
      opened = 1;
    }
    opens = opened != 0;
    x.h = h;
    x.t = t;
    x.flags = whole ? 4 : 0;
    x.slot = 2 * c + (head_item ? 0 : 1);
    int k;
    if (off < P) {
      x.branch = -1;
      x.lo = x.n = x.len = 0;
      k = off;
      count = P - off;
      keys_end = size;
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
      const int units_src = __shfl_sync(0xffffffffu, nu, src);
      k = s - (__shfl_sync(0xffffffffu, incl, src) - units_src);
      count = max(1, units_src - k);
      x.branch = bbase + src;
      x.lo = __shfl_sync(0xffffffffu, lo, src);
      x.n = __shfl_sync(0xffffffffu, n, src);
      x.len = __shfl_sync(0xffffffffu, len, src);
      keys_end = __shfl_sync(0xffffffffu, keys, src);
    }
    count = min(count, left);
    x.k0 = k * a.TN;
    x.nk = 0;
    off += count;
    left -= count;
    closes = left == 0 || off == units;
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
