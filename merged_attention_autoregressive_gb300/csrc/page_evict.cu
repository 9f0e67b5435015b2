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
// A cluster of CTAs shares a (branch, head): each reads, ranks and counts a part of
// its positions, sends its counts to the others' shared memory round by round and its
// words of kept rows at the end, and moves a part of the rows.  All of them have read
// the masses before any is overwritten.  None leaves while another may write to it:
// they agree first on status and length.
//
// What bounds it.  One row too many in 16 branches of 12 heads: a launch and three
// dependent reads, 8.8 us (5 us in a graph).  A frame of 1,560 rows over 4,680 in 4
// branches of 40 heads: 60 us, of which the rows' moves take 34 (HBM: 226 MB are
// 33 us), the reads of masses and stamps 4, the search 7, words and lists 7; the
// moves do not begin before the search ends, since all CTAs are resident at once.
// 29,000 rows down to 8,192 in the longest of 4 branches, 8 heads: 42 us, half of
// them its search and half its moves, on 32 of 152 SMs.
// Ranks and search made by each CTA of a cluster for itself: 63 and 54 us.  Counts
// exchanged by the cluster's own barrier: 64 and 46 us (a round costs 1,200 to 2,500
// cycles; messages and a barrier in shared memory cost 650).  Two bits a round: as
// fast as one, since the comparisons then bound it.  Clusters of 8 that are not all
// resident: 60 us for the long prompts.  Loads one after the other: 85 us for a frame;
// moves found bit by bit: 63 us for a long prompt.  Listing the values near the last
// kept one and searching among those alone after twelve bits gained nothing.
#include "common.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kList = 1024;  // moves listed at a time
constexpr int kMaxCluster = 8;
constexpr int kMostWords = (1 << 19) / 32;  // of 32 positions in a table (longer ones are refused)
// CTAs of an SM, by threads and integers of a thread.
__host__ __device__ constexpr int resident_of(int threads, int keys) { return threads == 1024 ? 1 : keys > 8 ? 3 : 4; }

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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of x (shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t address_at(const void* x, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(x)), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_at(uint32_t* x, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(address_at(x, rank)), "r"(v) : "memory");
}
// v to the place of x in CTA `rank`, which completes four bytes of its barrier.
__device__ __forceinline__ void send(int* x, uint64_t* bar, int rank, int v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(address_at(x, rank)),
               "r"(v), "r"(address_at(bar, rank))
               : "memory");
}
// Waits for what other CTAs of the cluster send; false when it has not come in 2 s.
__device__ __forceinline__ bool wait_sent(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < tc::kWaitPolls; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "n"(tc::kSuspendNs)
        : "memory");
    if (ok) return true;
  }
  return false;
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

// kKeys: integers in a thread's registers, for up to kThreads kKeys positions of a
// CTA; 0: they are made anew in every round (longer tables).  shares: a cluster of
// CTAs has the (branch, head).  per: 16-byte vectors of a row.
template <int kThreads, int kKeys, bool shares, int per>
__global__ void __launch_bounds__(kThreads, resident_of(kThreads, kKeys)) page_evict_kernel(const EvictArgs a, int32_t* st) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t words[];  // [words] kept, [words] ties, then counts
  __shared__ int sums[2][kWarps];
  __shared__ int told[2][kMaxCluster];         // counts of each CTA of the cluster
  __shared__ uint64_t heard[2];
  __shared__ int2 result;
  __shared__ uint32_t begins[kMaxCluster][3];  // what each of them starts from
  __shared__ int scan[33];
  __shared__ int src[kList], dst[kList];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / a.cluster, part = shares ? blockIdx.x % a.cluster : 0;
  const int b = item / a.H, h = item % a.H;
  const int32_t* const table = a.table + (size_t)b * a.max_pages;
  if (shares) {
    if (tid == 0) {
      tc::mbar_init(&heard[0], 1);
      tc::mbar_init(&heard[1], 1);
      tc::fence_mbar_init();
    }
    __syncwarp();
    cluster_arrive();  // this CTA's shared memory is there
  }
  pdl_wait();
  if (tid == 0) {
    const int n = a.len[b];
    begins[part][0] = n;
    begins[part][1] = a.born ? a.total[b] : n;
  }
  bool stop = block_status_bad(st);
  const int len = (int)begins[part][0], total = (int)begins[part][1];
  const bool fits = len >= 0 && (long long)len <= ((long long)a.max_pages << a.page_shift);
  if (shares) {
    // the CTAs of a cluster write to one another: all of them go on, or none
    cluster_wait();
    if (tid < a.cluster) {
      if (tid != part) {
        store_at(&begins[part][0], tid, (uint32_t)len);
        store_at(&begins[part][1], tid, (uint32_t)total);
      }
      store_at(&begins[part][2], tid, (uint32_t)stop);
    }
    __syncwarp();
    cluster_arrive();
  } else if (stop) {
    return;
  }
  // this CTA's positions: whole words of them
  const bool none = !fits || len <= a.budget;
  const int span = none ? 0 : shares ? (int)(((unsigned)len + 32u * a.cluster - 1) / (32u * a.cluster)) * 32 : len;
  const int lo = min(part * span, len), hi = none ? lo : min(lo + span, len);
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
  uint32_t* const kept = words;
  uint32_t* const tied = words + a.words;
  bool bad = false;
  // the ranks of positions lo + (i0 + i) kThreads + tid, their loads side by side
  auto keys_at = [&](int i0, auto many, uint32_t* key) {
    constexpr int n = decltype(many)::value;
    int row[n], age[n];
    float mass[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int p = lo + (i0 + i) * kThreads + tid;
      row[i] = p < hi ? row_of(a, table, h, p) : -1;
      bad = bad || (p < hi && row[i] < 0);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      age[i] = row[i] >= 0 && a.born ? a.born[row[i]] : lo + (i0 + i) * kThreads + tid;
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
  const int rounds = (hi - lo + kThreads - 1) / kThreads;
  if (kKeys) {
#pragma unroll
    for (int i = 0; i < kKeys; i += 8)
      if (i == 0 || i < rounds) {
        keys_at(i, std::integral_constant<int, 8>(), key + i);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) key[i + e] = 0u;
      }
  }
  if (shares) {
    cluster_wait();
    for (int r = 0; r < a.cluster; ++r)
      stop = stop || begins[r][2];
    if (stop) return;
    for (int r = 0; r < a.cluster; ++r) stop = stop || (int)begins[r][0] != len || (int)begins[r][1] != total;
    if (stop) {  // the lengths are being written meanwhile
      if (tid == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
      return;
    }
  }
  if (!fits) {
    if (tid == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
    return;
  }
  if (none) {
    if (a.copies) copy(len, [](int) { return true; });
    return;
  }
  const int nw = (len + 31) / 32;
  // how many values of the (branch, head) are at least `least`, for every thread.  A
  // turn's counts have been read before those of the turn after the next can come:
  // each CTA sends that one's when it has the next turn's of all.
  int turn = 0;
  bool ok = true;
  auto count = [&](uint32_t least) {
    int c = 0;
    if (kKeys) {
#pragma unroll
      for (int i = 0; i < kKeys; i += 8)
        if (i == 0 || i < rounds)
#pragma unroll
          for (int e = 0; e < 8; ++e) c += key[i + e] >= least;
    } else {
      for (int i = 0; i < rounds; ++i) c += key_at(i) >= least;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    const int at = turn & 1, parity = turn >> 1 & 1;
    ++turn;
    if (lane == 0) sums[at][warp] = c;
    __syncthreads();
    if (!shares) return __reduce_add_sync(0xffffffffu, lane < kWarps ? sums[at][lane] : 0);
    if (warp == 0) {
      c = __reduce_add_sync(0xffffffffu, lane < kWarps ? sums[at][lane] : 0);
      if (lane == 0) tc::mbar_arrive_expect_tx(&heard[at], a.cluster * 4);
      __syncwarp();
      if (lane < a.cluster) send(&told[at][part], &heard[at], lane, c);
      __syncwarp();
      const bool came = __all_sync(0xffffffffu, wait_sent(&heard[at], parity));
      c = __reduce_add_sync(0xffffffffu, lane < a.cluster ? told[at][lane] : 0);
      if (lane == 0) result = make_int2(c, came);
    }
    __syncthreads();
    const int2 r = result;
    ok = ok && r.y;
    return r.x;
  };
  // the last kept value: the largest that at least `budget` values reach (rows
  // behind the length have the smallest value and come last among its ties)
  uint32_t last = 0u;
  bool exact = false;  // exactly `budget` values reach it
  if (a.budget == 0) {
    last = 0xffffffffu;
  } else {
    for (uint32_t bit = 0x80000000u; bit && !exact && ok; bit >>= 1) {
      const int c = count(last | bit);
      if (c >= a.budget) {
        last |= bit;
        exact = c == a.budget;
      }
    }
  }
  // how many of the ties at it stay
  int quota = a.budget;
  if (!exact && ok && last != 0xffffffffu) quota -= count(last + 1);
  auto mark = [&](int i, uint32_t k) {
    uint32_t more = __ballot_sync(0xffffffffu, k > last), ties = __ballot_sync(0xffffffffu, k == last);
    const int w = (lo >> 5) + i * kWarps + warp, live = hi - w * 32;
    if (live <= 0) return;
    if (live < 32) ties &= (1u << live) - 1u;
    if (exact) more |= ties;
    if (shares) {
      if (lane < a.cluster) {
        store_at(kept + w, lane, more);
        if (!exact) store_at(tied + w, lane, ties);
      }
    } else if (lane == 0) {
      kept[w] = more;
      tied[w] = ties;
    }
  };
  if (kKeys) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (i < rounds) mark(i, key[i]);
  } else {
    for (int i = 0; i < rounds; ++i) mark(i, key_at(i));
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  // (all masses of the (branch, head) are read before any is overwritten)
  if (shares) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (!ok) {
      if (tid == 0) status_set(st, FASTAR_ERR_TIMEOUT);
      return;
    }
  } else {
    __syncthreads();
  }
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
  // this CTA's share of the moves
  const int end = (int)((long long)moves * (part + 1) / a.cluster);
  for (int m0 = (int)((long long)moves * part / a.cluster); m0 < end; m0 += kList) {
    const int some = min(kList, end - m0);
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
    for (int i = tid; i < some; i += kThreads) {
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
    }
    __syncthreads();
    // the masses and stamps that move are on their way while the rows do
    float mass[kList / kThreads];
    int age[kList / kThreads];
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
      const int i = tid + k * kThreads;
      const bool there = i < some && src[i] >= 0;
      mass[k] = there ? a.mass[src[i]] : 0.f;
      age[k] = there && a.born ? a.born[src[i]] : 0;
    }
    constexpr int kAhead = 8;
    for (int e0 = tid; e0 < some * 2 * per; e0 += kThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int e = e0 + q * kThreads, i = e / (2 * per), c = e % (2 * per);
        if (e < some * 2 * per && src[i] >= 0) v[q] = __ldcs((c < per ? a.K : a.V) + (size_t)src[i] * per + c % per);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int e = e0 + q * kThreads, i = e / (2 * per), c = e % (2 * per);
        if (e < some * 2 * per && src[i] >= 0) __stcs((c < per ? a.K : a.V) + (size_t)dst[i] * per + c % per, v[q]);
      }
    }
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
      const int i = tid + k * kThreads;
      if (i < some && src[i] >= 0) {
        a.out_mass[dst[i]] = mass[k];
        if (a.born) a.out_born[dst[i]] = age[k];
      }
    }
    __syncthreads();
  }
  if (a.copies) copy(a.budget, [&](int p) { return kept[p >> 5] >> (p & 31) & 1u; });
  pdl_trigger();
}

template <int kThreads, int kKeys, bool shares>
int launch_keys(const EvictArgs& a, int items, int per, int32_t* st, cudaStream_t s) {
  auto kernel = per == 8    ? page_evict_kernel<kThreads, kKeys, shares, 8>
                : per == 16 ? page_evict_kernel<kThreads, kKeys, shares, 16>
                            : page_evict_kernel<kThreads, kKeys, shares, 32>;
  const int smem = 2 * a.words * 4;
  // The limit belongs to the kernel, not to this launch: another host thread's call may
  // set it between the two, so all calls set the same.
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMostWords * 4) != cudaSuccess) {
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
  cfg.numAttrs = shares ? 2 : 1;
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
  // CTAs of a (branch, head): as many as are resident at once and have 64 rows each
  // to move, or eight values a thread to search, if the tables are as long as they
  // may be
  const int threads = room <= 8192 ? 256 : 1024, moves = min(budget, room - budget);
  int keys = (room + threads - 1) / threads;
  a.cluster = 1;
  while (a.cluster < kMaxCluster && (128 * a.cluster <= moves || keys > 8)) {
    const int next = 2 * a.cluster, fewer = (room + next * threads - 1) / (next * threads);
    if (next * items > 152 * resident_of(threads, fewer)) break;
    a.cluster = next;
    keys = fewer;
  }
  if (a.cluster == 1) {
    if (keys <= 8) return launch_keys<256, 8, false>(a, items, per, st, s);
    if (threads == 256) return launch_keys<256, 32, false>(a, items, per, st, s);
    if (keys <= 32) return launch_keys<1024, 32, false>(a, items, per, st, s);
    return launch_keys<1024, 0, false>(a, items, per, st, s);
  }
  if (threads == 256) {
    if (keys <= 8) return launch_keys<256, 8, true>(a, items, per, st, s);
    return launch_keys<256, 16, true>(a, items, per, st, s);
  }
  if (keys <= 8) return launch_keys<1024, 8, true>(a, items, per, st, s);
  if (keys <= 16) return launch_keys<1024, 16, true>(a, items, per, st, s);
  return launch_keys<1024, 0, true>(a, items, per, st, s);
}

}  // namespace fastar
