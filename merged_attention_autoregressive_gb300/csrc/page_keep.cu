// fastar_page_keep: the new tokens of a branch that stay move to the front of
// the new positions, in order (the accepted path of a tree of drafts).
//
// Token j that stays moves from position past + r_j to past + j, where r_j >= j
// ascends.  In place: a row is written only where every row that still has to be
// read lies behind, so a chunk of ascending tokens is read into registers, the
// threads of the (branch, head) meet, and the chunk is written.
//
// A CTA takes 128 bytes or less of every row of a (branch, head): columns do not
// meet, so that is where the work is split when rows are long or heads few.  The
// next chunk is read before the present one is written, for its rows lie behind all
// of those.
//
// What bounds it: memory where many rows move (half of 4 x 4,680 tokens of 12 heads:
// 28 us, 4.1 TB/s; 100 us with chunks of 64 rows, one after the other; chunks of 512
// rows 40 us, ids read two chunks ahead 30 us), a launch and
// four dependent reads (offsets, ids, pages, rows) where a path of a few drafts does
// (6 of 31 drafts of 16 branches: 4.6 us, 3.3 us in a graph).
#include "common.cuh"

namespace fastar {
namespace {

constexpr int kVecs = 4;   // 16-byte vectors of a thread in a chunk

struct KeepArgs {
  const int32_t* cu;
  const int32_t* rows;
  const int32_t* cu_keep;
  const int32_t* len;
  const int32_t* table;
  uint4* K;
  uint4* V;
  int M, H, max_pages, page_shift, n_pages, per;  // per: 16-byte vectors of a row
};

// Row of position p of branch b and head h in the pages; -1: there is none.
__device__ __forceinline__ int row_of(const KeepArgs& a, int b, int h, int p) {
  const int i = p >> a.page_shift;
  if (p < 0 || i >= a.max_pages) return -1;
  const int id = a.table[(size_t)b * a.max_pages + i];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((id * a.H + h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

// grid (H slices, B, keys and values); kSlice: vectors of a row in a CTA.
template <int kThreads, int kSlice>
__global__ void __launch_bounds__(kThreads) page_keep_kernel(const KeepArgs a, int32_t* st) {
  pdl_wait();
  const int b = blockIdx.y, slices = a.per / kSlice, h = blockIdx.x / slices, slice = blockIdx.x - h * slices;
  uint4* const x = (blockIdx.z ? a.V : a.K) + slice * kSlice + threadIdx.x % kSlice;
  if (block_status_bad(st)) return;
  const int lo = a.cu[b], hi = a.cu[b + 1], k0 = a.cu_keep[b], k1 = a.cu_keep[b + 1], len = a.len[b];
  const long long room = (long long)a.max_pages << a.page_shift;
  const bool ok = lo >= 0 && hi >= lo && (b != 0 || lo == 0) && k0 >= 0 && k1 >= k0 && k1 <= a.M &&
                  (b != 0 || k0 == 0) && k1 - k0 <= hi - lo && len >= 0 && len <= room;
  if (!ok && threadIdx.x == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (!ok) return;
  const int past = len - (hi - lo), n = k1 - k0;  // (past may be negative: those positions have no row)
  constexpr int kRows = kThreads / kSlice;        // rows of one vector per thread
  const int t = threadIdx.x / kSlice;
  // where the vectors of the chunk from j0 on are and where they go (-1: nowhere)
  auto place = [&](int j0, int (&from)[kVecs], int (&to)[kVecs]) {
    int r[kVecs], before[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
      const int j = j0 + e * kRows + t;
      r[e] = j < n ? a.rows[k0 + j] : -1;
      before[e] = j < n && j > 0 ? a.rows[k0 + j - 1] : lo - 1;
    }
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
      const int j = j0 + e * kRows + t;
      const bool fine = r[e] > before[e] && r[e] >= lo && r[e] < hi, moves = j < n && fine && r[e] - lo != j;
      if (j < n && !fine) status_set(st, FASTAR_ERR_DEVICE_ARG);
      from[e] = moves ? row_of(a, b, h, past + r[e] - lo) : -1;
      to[e] = moves ? row_of(a, b, h, past + j) : -1;
      if (moves && (from[e] < 0 || to[e] < 0)) {
        status_set(st, FASTAR_ERR_DEVICE_ARG);
        to[e] = -1;
      }
    }
  };
  constexpr int kChunk = kRows * kVecs;
  int from[kVecs], to[kVecs];
  uint4 v[kVecs];
  auto read = [&](uint4 (&v)[kVecs]) {
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
      if (to[e] >= 0) v[e] = __ldcs(x + (size_t)from[e] * a.per);
  };
  place(0, from, to);
  read(v);
  for (int j0 = 0; j0 < n; j0 += kChunk) {
    int at[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) at[e] = to[e];
    uint4 next[kVecs];
    if (j0 + kChunk < n) {
      place(j0 + kChunk, from, to);
      read(next);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
      if (at[e] >= 0) __stcs(x + (size_t)at[e] * a.per, v[e]);
#pragma unroll
    for (int e = 0; e < kVecs; ++e) v[e] = next[e];
  }
  pdl_trigger();
}

}  // namespace

int launch_page_keep(const fastar_pages* pg, const int32_t* cu, const int32_t* rows, int M,
                     const int32_t* cu_keep, int32_t* st, cudaStream_t s) {
  KeepArgs a = {cu, rows, cu_keep, pg->len, pg->table, (uint4*)pg->K, (uint4*)pg->V, M, pg->H,
                pg->max_pages, 0, pg->n_pages, pg->D * (pg->dt == FASTAR_BF16 ? 2 : 4) / 16};
  while ((1 << a.page_shift) < pg->page) ++a.page_shift;
  // 128-byte slices, chunks of 64 rows for a path of drafts; of 256 rows where a branch
  // keeps many, by 256 threads in slices of 64 bytes (half of 4 x 4,680 tokens of 12
  // heads: 28 us, 30 us by 512 threads in slices of 128; 16 branches of 40 heads: 272
  // and 267 us), or by 512 in slices of 64 or 32 where that leaves SMs without a CTA
  // (5,550 of 6,142 tokens of one branch, 4 heads of 512 bytes: 16 us, 37 us at 128
  // bytes)
  cudaError_t rc;
  auto launch = [&](auto kernel, int threads, int slice) {
    rc = launch_pdl(kernel, dim3(a.H * (a.per / slice), pg->B, 2), dim3(threads), 0, s, a, st);
  };
  const long long ctas = 2ll * pg->B * a.H * a.per;
  if (M <= 128ll * pg->B)
    launch(page_keep_kernel<128, 8>, 128, 8);
  else if (ctas / 8 >= 152)
    launch(page_keep_kernel<256, 4>, 256, 4);
  else if (ctas / 4 >= 152)
    launch(page_keep_kernel<512, 4>, 512, 4);
  else
    launch(page_keep_kernel<512, 2>, 512, 2);
  if (rc != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_keep");
  return FASTAR_OK;
}

}  // namespace fastar
