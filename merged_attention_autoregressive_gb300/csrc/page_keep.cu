// fastar_page_keep: the new tokens of a branch that stay move to the front of
// the new positions, in order (the accepted path of a tree of drafts).
//
// Token j that stays moves from position past + r_j to past + j, where r_j >= j
// ascends.  In place: a row is written only where every row that still has to be
// read lies behind, so a chunk of ascending tokens is read into registers, the
// threads of the (branch, head) meet, and the chunk is written.
//
// What bounds it: memory where many rows move, a launch and three dependent
// reads (offsets, page ids, rows) where a path of a few drafts does.
#include "common.cuh"

namespace fastar {
namespace {

constexpr int kThreads = 256, kVecs = 4;  // 16-byte vectors in flight per thread

struct KeepArgs {
  const int32_t* cu;
  const int32_t* rows;
  const int32_t* cu_keep;
  const int32_t* len;
  const int32_t* table;
  uint4* K;
  uint4* V;
  int M, H, max_pages, page_shift, n_pages;
};

// Row of position p of branch b and head h in the pages; -1: there is none.
__device__ __forceinline__ int row_of(const KeepArgs& a, int b, int h, int p) {
  const int i = p >> a.page_shift;
  if (p < 0 || i >= a.max_pages) return -1;
  const int id = a.table[(size_t)b * a.max_pages + i];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((id * a.H + h) << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

// grid (H, B, keys and values); per: 16-byte vectors of a row.
template <int per>
__global__ void __launch_bounds__(kThreads) page_keep_kernel(const KeepArgs a, int32_t* st) {
  pdl_wait();
  const int b = blockIdx.y, h = blockIdx.x;
  uint4* const x = blockIdx.z ? a.V : a.K;
  if (block_status_bad(st)) return;
  const int lo = a.cu[b], hi = a.cu[b + 1], k0 = a.cu_keep[b], k1 = a.cu_keep[b + 1], len = a.len[b];
  const long long room = (long long)a.max_pages << a.page_shift;
  const bool ok = lo >= 0 && hi >= lo && (b != 0 || lo == 0) && k0 >= 0 && k1 >= k0 && k1 <= a.M &&
                  (b != 0 || k0 == 0) && k1 - k0 <= hi - lo && len >= 0 && len <= room;
  if (!ok && threadIdx.x == 0) status_set(st, FASTAR_ERR_DEVICE_ARG);
  if (!ok) return;
  const int past = len - (hi - lo), n = k1 - k0;  // (past may be negative: those positions have no row)
  constexpr int kRows = kThreads / per;  // rows of one vector per thread
  const int c = threadIdx.x % per, t = threadIdx.x / per;
  for (int j0 = 0; j0 < n; j0 += kRows * kVecs) {
    uint4 v[kVecs];
    int to[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
      const int j = j0 + e * kRows + t;
      to[e] = -1;
      if (j >= n) continue;
      const int r = a.rows[k0 + j], before = j > 0 ? a.rows[k0 + j - 1] : lo - 1;
      if (r <= before || r < lo || r >= hi) {
        status_set(st, FASTAR_ERR_DEVICE_ARG);
        continue;
      }
      if (r - lo == j) continue;  // it stays where it is
      const int from = row_of(a, b, h, past + r - lo);
      to[e] = row_of(a, b, h, past + j);
      if (from < 0 || to[e] < 0) {
        status_set(st, FASTAR_ERR_DEVICE_ARG);
        to[e] = -1;
        continue;
      }
      v[e] = x[(size_t)from * per + c];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
      if (to[e] >= 0) x[(size_t)to[e] * per + c] = v[e];
  }
  pdl_trigger();
}

}  // namespace

int launch_page_keep(const fastar_pages* pg, const int32_t* cu, const int32_t* rows, int M,
                     const int32_t* cu_keep, int32_t* st, cudaStream_t s) {
  KeepArgs a = {cu, rows, cu_keep, pg->len, pg->table, (uint4*)pg->K, (uint4*)pg->V, M, pg->H,
                pg->max_pages, 0, pg->n_pages};
  while ((1 << a.page_shift) < pg->page) ++a.page_shift;
  const int per = pg->D * (pg->dt == FASTAR_BF16 ? 2 : 4) / 16;
  auto kernel = per == 8 ? page_keep_kernel<8> : per == 16 ? page_keep_kernel<16> : page_keep_kernel<32>;
  const cudaError_t rc = launch_pdl(kernel, dim3(a.H, pg->B, 2), dim3(kThreads), 0, s, a, st);
  if (rc != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "page_keep");
  return FASTAR_OK;
}

}  // namespace fastar
