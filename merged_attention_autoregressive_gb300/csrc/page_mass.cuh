// Work of fastar_page_mass, shared by its kernels.
//
// An item is a tile of TK positions of one branch and one key/value head.  Its
// rows are the queries of the branch's new tokens that see the tile, row r =
// token i0 + r / g, head h g + r % g, TQ of them at a time: the scores of a tile
// are summed over the rows, so an item is one pass over the queries with its keys
// held, and its masses are written once.  Items follow one another branch by
// branch, tile by tile, head by head (all heads of a page lie side by side, and
// the first tiles, which most tokens see, come first); CTA c takes the items c,
// c + G, c + 2 G, ...
//
// Where items do not fill the CTAs evenly, each item's rows are cut into `parts`
// runs of tiles; each leaves its sums in the workspace and
// page_mass_join adds them in order, so results do not change from run to run.
//
// The lengths live on the device: every CTA walks them, 32 branches at a time.
#pragma once

#include "branch.cuh"

namespace fastar {

struct MassArgs {
  const void* q;        // [Hq][N][D]
  const float* lse;     // [Hq][N]
  const int32_t* rows;  // [M] query row of each token, or null
  const int32_t* cu;    // [B + 1]
  const int32_t* len;   // [B]
  const int32_t* table;
  const void* K;
  float* mass;
  int32_t* born;        // or null
  const int32_t* total;
  int N, M, Hq, H, g, B, max_pages, page_shift, n_pages, block, G, split;
  int rows_lo, rows_hi;  // the kernel takes branches of rows_lo < n g <= rows_hi rows
  float scale, decay;
  float* part;          // [kMostParts G][TK] sums of cut items
};

constexpr int kMassFew = 32, kMassFew32 = 16;  // rows of a branch, for one head, that are a few: bf16, fp32

struct MassItem {
  int b, h, k0;    // branch, head, first position of the tile
  int lo, n, len;  // first token, tokens, length of the branch
  int i0;          // first token that sees the tile
};

// Row of position p in the pages of branch b, head h; -1: its page is not there.
__device__ __forceinline__ int mass_row(const MassArgs& a, int b, int h, int p) {
  const int id = a.table[(size_t)b * a.max_pages + (p >> a.page_shift)];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((id * a.H + h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

// Items of a call, and units of parts of them, fit an unsigned: more are refused.
constexpr long long kMaxItems = 1 << 30;

// A warp's place among the items; all lanes in step.
template <int TK>
struct MassWalk {
  unsigned base, total;   // items before the 32 branches, and of them
  unsigned mine, incl;    // lane: items of branch b0 + lane; items up to and with it
  int b0, lo, n, len;
  MassItem x;             // the item found last
  unsigned left;          // items behind it in its branch

  __device__ __forceinline__ long long load(const MassArgs& a, bool& ok) {
    const int lane = threadIdx.x & 31, b = b0 + lane;
    lo = n = len = 0;
    if (b < a.B) {
      lo = a.cu[b];
      const int hi = a.cu[b + 1];
      len = a.len[b];
      ok = ok && lo >= 0 && hi >= lo && hi <= a.M && (b != 0 || lo == 0) && len >= 0 &&
           (long long)len <= ((long long)a.max_pages << a.page_shift);
      n = ok ? hi - lo : 0;
      if (n * a.g <= a.rows_lo || n * a.g > a.rows_hi) n = 0;
    }
    const long long items = n > 0 ? (long long)(((unsigned)len + TK - 1u) / TK) * a.H : 0;
    ok = ok && items < kMaxItems / 32;
    mine = ok ? (unsigned)items : 0u;
    incl = (unsigned)warp_incl_scan((int)mine);
    total = __shfl_sync(0xffffffffu, incl, 31);
    return total;
  }
  // Items of the call, and the most tokens of a branch; ok: every length and
  // offset holds.
  __device__ __forceinline__ unsigned count(const MassArgs& a, int& most, bool& ok) {
    long long items = 0;
    most = 0;
    for (b0 = 0; b0 < a.B; b0 += 32) {
      items += load(a, ok);
      most = max(most, __reduce_max_sync(0xffffffffu, n));
    }
    ok = __all_sync(0xffffffffu, ok) && items < kMaxItems;
    base = 0;
    b0 = 0;
    left = 0;
    if (a.B > 32) {
      bool same = true;
      load(a, same);
    } else if (a.B == 0) {
      total = 0;
    }
    return ok ? (unsigned)items : 0u;
  }
  // Item `it`, at or behind the last one asked for.
  __device__ __forceinline__ const MassItem& find(const MassArgs& a, unsigned it) {
    while (it >= base + total) {
      base += total;
      b0 += 32;
      bool ok = true;
      load(a, ok);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, base + incl > it)) - 1;
    const unsigned off = it - base - __shfl_sync(0xffffffffu, incl - mine, src);
    left = __shfl_sync(0xffffffffu, mine, src) - off - 1u;
    x.b = b0 + src;
    const unsigned tile = off / (unsigned)a.H;
    x.h = (int)(off - tile * (unsigned)a.H);
    x.k0 = (int)tile * TK;
    x.lo = __shfl_sync(0xffffffffu, lo, src);
    x.n = __shfl_sync(0xffffffffu, n, src);
    x.len = __shfl_sync(0xffffffffu, len, src);
    first_token(a);
    return x;
  }
  // The item `by` behind the last one, or `it` where that is another's (the same
  // item, found without a search while the branch has as many: with one unit per
  // item the search is what every warp would do most of the time).  by_tiles, by_heads:
  // by / H and by % H.
  __device__ __forceinline__ const MassItem& next(const MassArgs& a, unsigned it, unsigned by, int by_tiles, int by_heads) {
    if (by > left) return find(a, it);
    left -= by;
    x.h += by_heads;
    x.k0 += by_tiles * TK;
    if (x.h >= a.H) {
      x.h -= a.H;
      x.k0 += TK;
    }
    first_token(a);
    return x;
  }
  // the first token whose last block reaches the tile
  __device__ __forceinline__ void first_token(const MassArgs& a) {
    x.i0 = a.block > 0 ? min(x.n, max(0, x.k0 / a.block * a.block - (x.len - x.n))) : 0;
  }
};

// Tiles of TQ rows of an item that `tokens` tokens see.  On the tensor cores
// (TQ 128) the rows of many tokens that lie in order go head by head, so that a
// tile is one run of memory; otherwise a token's heads follow one another and few
// tokens fill few tiles.
__device__ __forceinline__ bool mass_by_head(const MassArgs& a, int tokens, int TQ) {
  return TQ == 128 && !a.rows && tokens >= 64;
}
__device__ __forceinline__ int mass_tiles(const MassArgs& a, int tokens, int TQ) {
  return mass_by_head(a, tokens, TQ) ? (tokens + TQ - 1) / TQ * a.g : (tokens * a.g + TQ - 1) / TQ;
}

// Whether items may be cut: where a branch can be expected to have rows for two
// tiles (the join's launch for nothing costs 2 us of a small call).
inline bool mass_split(const MassArgs& a, int TQ) { return (long long)a.M * a.g > TQ + 4ll * a.B; }

// Parts of each item (whole warp): the number that makes the fullest CTA's share
// least, in tiles of rows, of which an item's begin and end cost about one more
// and the join's launch three.
constexpr int kMostParts = 8;  // parts per CTA
__device__ __forceinline__ int mass_parts(const MassArgs& a, unsigned items, int most, int TQ) {
  const unsigned G = a.G;
  if (!a.split || items == 0 || items > G * kMostParts / 2) return 1;
  const unsigned tiles = mass_tiles(a, most, TQ), limit = min(tiles, G * kMostParts / items);
  unsigned best = 0xffffffffu, at = 1;
  for (unsigned p = 1 + (threadIdx.x & 31); p <= limit; p += 32) {
    const unsigned cost = (items * p + G - 1) / G * ((tiles + p - 1) / p + 1) + (p > 1 ? 3 : 0);
    if (cost < best) {
      best = cost;
      at = p;
    }
  }
  const unsigned least = __reduce_min_sync(0xffffffffu, best);
  return (int)__reduce_min_sync(0xffffffffu, best == least ? at : 0xffffffffu);
}

// Tiles t0 .. t1 - 1 of an item's are those of part `part`.
__device__ __forceinline__ void mass_share(int tiles, unsigned part, unsigned parts, int& t0, int& t1) {
  t0 = 0;
  t1 = tiles;
  if (parts > 1) {
    const unsigned each = (unsigned)tiles / parts, more = (unsigned)tiles - each * parts;
    t0 = (int)(part * each + min(part, more));
    t1 = t0 + (int)(each + (part < more ? 1u : 0u));
  }
}

// The mass of a position with what it drew in this call, and its token's number.
__device__ __forceinline__ void mass_write(const MassArgs& a, int b, int past, int len, int p, int row, float old, float drew) {
  a.mass[row] = p >= past ? drew : fmaf(a.decay, old, drew);
  if (a.born && p >= past) a.born[row] = a.total[b] - len + p;
}

int launch_mass_few(int D, bool bf16, MassArgs a, int32_t* st, cudaStream_t s);
int launch_mass_tc(int D, MassArgs a, int32_t* st, cudaStream_t s);
int launch_mass_join(int TK, int TQ, const MassArgs& a, int32_t* st, cudaStream_t s);

}  // namespace fastar
