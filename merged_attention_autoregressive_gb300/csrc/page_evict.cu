// fastar_page_evict: every branch and head keeps `budget` of its rows, those
// that drew the most attention beside the first and the latest ones.
//
// The kept rows are the largest by (protected, mass, lower position first).  A
// mass is compared as an unsigned integer of the same order, so the last kept
// value is found bit by bit from the top: a bit stays set while at least `budget`
// values reach the candidate, and the search ends as soon as exactly `budget` do.
// The integers of a (branch, head) stay in registers over the rounds, a round is
// a count over the CTA.  Ties at the last value go to the lower positions by a
// prefix sum over words of 32 positions.  Kept rows from the budget on then move
// into the holes before it, both in ascending order: sources and targets are
// disjoint, rows below the budget that stay are not touched, and as few rows move
// as can.
//
// A cluster of CTAs shares the moves of a (branch, head); each of its CTAs does
// the selection for itself (a reduction across CTAs costs more than it saves) and
// all of them have read the masses before any is overwritten.
//
// What bounds it.  One row too many in 16 branches of 12 heads: a launch and three
// dependent reads, 8.6 us (5 us in a graph).  A frame of 1,560 rows over 4,680 in 4
// branches of 40 heads: 63 us, of which the moves take 33 (HBM: 226 MB are 33 us),
// the reads of masses and stamps 9, the search 8, the rest words, lists and the
// masses' own moves; the two halves do not overlap, since all CTAs are resident at
// once.  29,000 rows down to 8,192 in the longest of 4 branches, 8 heads: 54 us, the
// search 17 of them (25 rounds over 29 integers of each of 1,024 threads).  Loads one
// after the other cost a frame 85 us, moves found bit by bit a long prompt 63 us.
// Listing the values near the last kept one and searching among those alone after
// twelve bits gained nothing.
#include "common.cuh"

namespace fastar {
namespace {

constexpr int kList = 1024;  // moves listed at a time

struct EvictArgs {
  const int32_t* len;
  const int32_t* table;
  uint4* K;
  uint4* V;
  const float* mass;
  const int32_t* born;   // or null: positions tell the age
  const int32_t* total;
  float* out_mass;       // may be mass and born
  int32_t* out_born;
  int H, max_pages, page_shift, n_pages, budget, first, recent, cluster, words, copies;
};

__device__ __forceinline__ int row_of(const EvictArgs& a, const int32_t* table, int h, int p) {
  const int id = table[p >> a.page_shift];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((id * a.H + h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

// The order of the rows as an unsigned integer: protected rows first, then by
// mass; a mass that is not a number comes last.
__device__ __forceinline__ uint32_t rank_of(const EvictArgs& a, int age, float mass, int total) {
  if (age < a.first || age >= total - a.recent) return 0xffffffffu;
  const float x = mass + 0.f;  // one zero
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The lowest n set bits of w.
__device__ __forceinline__ uint32_t lowest(uint32_t w, int n) {
  if (n <= 0) return 0u;
  if (n >= __popc(w)) return w;
  uint32_t r = 0;
  for (; n > 0; --n) {
    r |= w & (0u - w);
    w &= w - 1;
  }
  return r;
}

// Each thread's count summed over the CTA (one barrier; sum[round & 1] is in use).
template <int kWarps>
__device__ __forceinline__ int block_count(int c, int (*sum)[kWarps], int round) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) sum[round & 1][threadIdx.x >> 5] = c;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < kWarps ? sum[round & 1][threadIdx.x & 31] : 0);
}

// kKeys: integers in a thread's registers, for up to kThreads kKeys positions; 0:
// they are made anew in every round (longer tables).  per: 16-byte vectors of a row.
template <int kThreads, int kKeys, int per>
__global__ void __launch_bounds__(kThreads, kThreads == 1024 ? 1 : kKeys > 8 ? 3 : 4)
    page_evict_kernel(const EvictArgs a, int32_t* st) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t words[];  // [words] kept, [words] ties, then counts
  __shared__ int sum[2][kWarps], scan[33];
  __shared__ int src[kList], dst[kList];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / a.cluster, part = blockIdx.x % a.cluster;
  const int b = item / a.H, h = item % a.H;
  const int32_t* const table = a.table + (size_t)b * a.max_pages;
  const int len = a.len[b], total = a.born ? a.total[b] : len;
  // (a CTA that has left does not hold up its cluster's barrier)
  if (block_status_bad(st)) return;
  if (len < 0 || (long long)len > ((long long)a.max_pages << a.page_shift)) {
    if (tid == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    return;
  }
  // masses and stamps of the positions below n that stay, four at a time
  auto copy = [&](int n, auto stays) {
    for (int p0 = part * kThreads + tid; p0 < n; p0 += 4 * a.cluster * kThreads) {
      int row[4], age[4];
      float mass[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + i * a.cluster * kThreads;
        row[i] = p < n && stays(p) ? row_of(a, table, h, p) : -2;
        if (row[i] == -1) status_set(st, FASTAR_ERR_DEVICE_ARG);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mass[i] = row[i] >= 0 ? a.mass[row[i]] : 0.f;
        age[i] = row[i] >= 0 && a.born ? a.born[row[i]] : 0;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row[i] >= 0) {
          a.out_mass[row[i]] = mass[i];
          if (a.born) a.out_born[row[i]] = age[i];
        }
    }
  };
  if (len <= a.budget) {
    if (a.copies) copy(len, [](int) { return true; });
    return;
  }
  uint32_t* const kept = words;
  uint32_t* const tied = words + a.words;
  const int nw = (len + 31) / 32;
  bool bad = false;
  // the ranks of positions (i0 + i) kThreads + tid, their loads side by side
  auto keys_at = [&](int i0, auto many, uint32_t* key) {
    constexpr int n = decltype(many)::value;
    int row[n], age[n];
    float mass[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int p = (i0 + i) * kThreads + tid;
      row[i] = p < len ? row_of(a, table, h, p) : -1;
      bad = bad || (p < len && row[i] < 0);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      age[i] = row[i] >= 0 && a.born ? a.born[row[i]] : (i0 + i) * kThreads + tid;
      mass[i] = row[i] >= 0 ? a.mass[row[i]] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) key[i] = row[i] >= 0 ? rank_of(a, age[i], mass[i], total) : 0u;
  };
  auto key_at = [&](int i) {
    uint32_t k;
    keys_at(i, std::integral_constant<int, 1>(), &k);
    return k;
  };
  uint32_t key[kKeys ? kKeys : 1];
  const int rounds = kKeys ? kKeys : (len + kThreads - 1) / kThreads;
  if (kKeys) {
#pragma unroll
    for (int i = 0; i < kKeys; i += 8)
      if (i == 0 || i * kThreads < len) {
        keys_at(i, std::integral_constant<int, 8>(), key + i);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) key[i + e] = 0u;
      }
  }
  auto count = [&](uint32_t least) {
    int c = 0;
    if (kKeys) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) c += key[i] >= least;
    } else {
      for (int i = 0; i < rounds; ++i) c += key_at(i) >= least;
    }
    return c;
  };
  // the last kept value: the largest that at least `budget` values reach (rows
  // behind the length have the smallest value and come last among its ties)
  uint32_t last = 0u;
  bool exact = false;  // exactly `budget` values reach it
  int round = 0;
  if (a.budget == 0) {
    last = 0xffffffffu;
  } else {
    for (uint32_t bit = 0x80000000u; bit && !exact; bit >>= 1) {
      const int c = block_count<kWarps>(count(last | bit), sum, round++);
      if (c >= a.budget) {
        last |= bit;
        exact = c == a.budget;
      }
    }
  }
  // how many of the ties at it stay
  int quota = 0x7fffffff;
  if (!exact && a.budget > 0)
    quota = a.budget - (last == 0xffffffffu ? 0 : block_count<kWarps>(count(last + 1), sum, round++));
  else if (a.budget == 0)
    quota = 0;
  auto mark = [&](int i, uint32_t k) {
    const uint32_t more = __ballot_sync(0xffffffffu, k > last), same = __ballot_sync(0xffffffffu, k == last);
    const int w = i * kWarps + warp;
    if (lane == 0 && w < nw) {
      const int live = len - w * 32;
      kept[w] = more;
      tied[w] = live >= 32 ? same : same & ((1u << live) - 1u);
    }
  };
  if (kKeys) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) mark(i, key[i]);
  } else {
    for (int i = 0; i < rounds; ++i) mark(i, key_at(i));
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  __syncthreads();
  // the ties that stay, in order
  if (!exact) {
    int carry = 0;
    for (int w0 = 0; w0 < nw; w0 += kThreads) {
      const int w = w0 + tid;
      const uint32_t t = w < nw ? tied[w] : 0u;
      int all;
      const int before = carry + block_excl_scan(__popc(t), scan, &all);
      if (w < nw) kept[w] |= lowest(t, quota - before);
      carry += all;
    }
    __syncthreads();
  } else {
    for (int w = tid; w < nw; w += kThreads) kept[w] |= tied[w];
    __syncthreads();
  }
  // how many holes (before the budget) or moving rows (behind its word) are in the
  // words before each; there are as many of them as of the others
  const int edge = a.budget >> 5;  // the word of the budget's own position
  const uint32_t below = (1u << (a.budget & 31)) - 1u;
  const int first_moves = __popc(kept[edge] & ~below);
  int all_words = 0;
  for (int w0 = 0; w0 < nw; w0 += kThreads) {
    const int w = w0 + tid;
    const uint32_t k = w < nw ? kept[w] : 0u;
    const int n = w >= nw ? 0 : w < edge ? __popc(~k) : w == edge ? __popc(~k & below) : __popc(k);
    int all;
    const int before = all_words + block_excl_scan(n, scan, &all);
    if (w < nw) tied[w] = before;
    all_words += all;
  }
  const int moves = (all_words + first_moves) / 2;
  __syncthreads();
  if (a.cluster > 1) cluster_sync();
  if (a.copies) copy(a.budget, [&](int p) { return kept[p >> 5] >> (p & 31) & 1u; });
  // this CTA's share of the moves
  const int end = (int)((long long)moves * (part + 1) / a.cluster);
  for (int m0 = (int)((long long)moves * part / a.cluster); m0 < end; m0 += kList) {
    const int n = min(kList, end - m0);
    // move m: the m-th hole and the m-th moving row, found among the words' counts
    auto find = [&](int m, int w0, int w1, int less) {  // last word of w0 .. w1 - 1 whose count is <= m
      while (w1 - w0 > 1) {
        const int mid = (w0 + w1) >> 1;
        if ((int)tied[mid] - less <= m)
          w0 = mid;
        else
          w1 = mid;
      }
      return w0;
    };
    auto nth = [](uint32_t bits, int k) {  // place of the k-th set bit
      int at = 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const int c = __popc(bits & ((1u << o) - 1u));
        if (k >= c) {
          k -= c;
          bits >>= o;
          at += o;
        }
      }
      return at;
    };
    for (int i = tid; i < n; i += kThreads) {
      const int m = m0 + i, less = moves - first_moves;
      const int w = find(m, 0, edge + 1, 0);
      const int to = w * 32 + nth(w < edge ? ~kept[w] : ~kept[w] & below, m - (int)tied[w]);
      // (the edge's own moving rows come before those of the words behind it)
      const int y = m < first_moves ? edge : find(m, edge + 1, nw, less);
      const int from = y * 32 + nth(y > edge ? kept[y] : kept[y] & ~below, y > edge ? m - ((int)tied[y] - less) : m);
      const int s = row_of(a, table, h, from), d = row_of(a, table, h, to);
      const bool there = s >= 0 && d >= 0;
      src[i] = there ? s : -1;
      dst[i] = d;
      if (there) {
        a.out_mass[d] = a.mass[s];
        if (a.born) a.out_born[d] = a.born[s];
      }
    }
    __syncthreads();
    constexpr int kAhead = 8;
    for (int e0 = tid; e0 < n * 2 * per; e0 += kThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int e = e0 + q * kThreads, i = e / (2 * per), c = e % (2 * per);
        if (e < n * 2 * per && src[i] >= 0) v[q] = __ldcs((c < per ? a.K : a.V) + (size_t)src[i] * per + c % per);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int e = e0 + q * kThreads, i = e / (2 * per), c = e % (2 * per);
        if (e < n * 2 * per && src[i] >= 0) __stcs((c < per ? a.K : a.V) + (size_t)dst[i] * per + c % per, v[q]);
      }
    }
    __syncthreads();
  }
  pdl_trigger();
}

template <int kThreads, int kKeys>
int launch_keys(EvictArgs a, int items, int per, int32_t* st, cudaStream_t s) {
  auto kernel = per == 8    ? page_evict_kernel<kThreads, kKeys, 8>
                : per == 16 ? page_evict_kernel<kThreads, kKeys, 16>
                            : page_evict_kernel<kThreads, kKeys, 32>;
  const int smem = 2 * a.words * 4;
  // CTAs of a (branch, head): as many as are resident at once and have 64 rows each
  // to move, if the tables are as long as they may be
  const int resident = 152 * (kThreads == 1024 ? 1 : kKeys > 8 ? 3 : 4);
  const int room = a.max_pages << a.page_shift, moves = min(a.budget, room - a.budget);
  a.cluster = 1;
  while (a.cluster < 8 && 2 * a.cluster * items <= resident && 128 * a.cluster <= moves) a.cluster *= 2;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(items * a.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_evict");
  return FASTAR_OK;
}

}  // namespace

int launch_page_evict(const fastar_pages* pg, const fastar_mass* mass, int budget, int first, int recent,
                      const fastar_mass* out, int32_t* st, cudaStream_t s) {
  EvictArgs a = {};
  a.len = pg->len;
  a.table = pg->table;
  a.K = (uint4*)pg->K;
  a.V = (uint4*)pg->V;
  a.mass = mass->mass;
  a.born = mass->born;
  a.total = mass->total;
  a.out_mass = out ? out->mass : mass->mass;
  a.out_born = out ? out->born : mass->born;
  a.copies = a.out_mass != a.mass;
  a.H = pg->H;
  a.max_pages = pg->max_pages;
  a.n_pages = pg->n_pages;
  while ((1 << a.page_shift) < pg->page) ++a.page_shift;
  a.budget = budget;
  a.first = first;
  a.recent = recent;
  const int room = pg->max_pages * pg->page, items = pg->B * pg->H;
  a.words = (room + 31) / 32;
  const int per = pg->D * (pg->dt == FASTAR_BF16 ? 2 : 4) / 16;
  if (room <= 2048) return launch_keys<256, 8>(a, items, per, st, s);
  if (room <= 8192) return launch_keys<256, 32>(a, items, per, st, s);
  if (room <= 32768) return launch_keys<1024, 32>(a, items, per, st, s);
  return launch_keys<1024, 0>(a, items, per, st, s);
}

}  // namespace fastar
