// C ABI of the FAST-AR per-chunk attention path: argument checks, workspace
// sizing and dispatch to the kernels.  Nothing here allocates, frees or
// synchronises; every launch goes to the caller's stream.
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace fastar {
// Every compute call is an NVTX range named after it, so that a profiler's
// timeline shows which call launched which kernels (a no-op without one).
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};
static std::atomic<uint64_t> g_launches{0};

// launch timing: caller-created events, recorded after each launch
static std::mutex g_tmu;
static std::atomic<int> g_timing{0};
static cudaEvent_t* g_tev = nullptr;
static int g_tcap = 0, g_tn = 0;
static const char* g_tname[4096];

void after_launch(cudaStream_t s, const char* name) {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (!g_timing.load(std::memory_order_acquire)) return;
  std::lock_guard<std::mutex> lock(g_tmu);
  if (g_tev && g_tn < g_tcap && g_tn < 4096) {
    if (cudaEventRecord(g_tev[g_tn], s) == cudaSuccess) g_tname[g_tn++] = name;
    else (void)cudaGetLastError();
  }
}

int launch_hash_simt(fastar_dtype dt, const void* x, int H, int N, int D, const void* planes,
                     int T, int B, uint32_t* codes, int32_t* st, cudaStream_t s);
int launch_hash_tc(fastar_dtype dt, const void* x, int H, int N, int D, const void* planes,
                   int T, int B, uint32_t* codes, int32_t* st, cudaStream_t s);
int launch_hash_tc_many(fastar_dtype dt, int n, const void* const* xs, const int* Ns, uint32_t* const* codes,
                        int H, int D, const void* planes, int T, int B, int32_t* st, cudaStream_t s);
int launch_annca_simt(fastar_dtype dt, const void* q, const void* k_p, const void* v_p,
                      const int32_t* kept_idx, const int32_t* kept_cnt, int H, int F, int n_f, int P,
                      int D, float scale, void* out, int32_t* st, cudaStream_t s);
int launch_annca_tc(fastar_dtype dt, const void* q, const void* k_p, const void* v_p,
                    const int32_t* kept_idx, const int32_t* kept_cnt, int H, int F, int n_f, int P,
                    int D, float scale, void* out, void* ws, size_t ws_bytes, int32_t* st, cudaStream_t s);
size_t annca_tc_ws_bytes(int H, int F, int P, int D);
int launch_annsa_simt(fastar_dtype dt, const void* q, const uint32_t* q_codes, int Nq,
                      const fastar_cache* c, float scale, void* out, float* lse, int32_t* st,
                      cudaStream_t s);
int launch_annsa_tc(fastar_dtype dt, const void* q, const uint32_t* q_codes, const int32_t* q_perm,
                    const int32_t* q_offsets, int Nq, const fastar_cache* c, float scale, void* out,
                    float* lse, void* ws, int32_t* st, cudaStream_t s);
size_t annsa_tc_ws_bytes(int H, int Nq, int D, int T);
size_t annsa_parts_ws_bytes(int H, int Nq, int D, int parts);
int launch_annsa_parts(const void* q, const uint32_t* q_codes, const int32_t* q_perm, int Nq,
                       const fastar_cache* c, float scale, int base, int parts, void* ws, int32_t* st,
                       cudaStream_t s);
int launch_annsa_combine(int H, int Nq, int parts, const void* ws, void* out, float* lse, int32_t* st,
                         cudaStream_t s);

int launch_hash(fastar_dtype dt, const void* x, int H, int N, int D, const void* planes, int T,
                int B, uint32_t* codes, int32_t* st, cudaStream_t s) {
  int rc = launch_hash_tc(dt, x, H, N, D, planes, T, B, codes, st, s);
  if (rc != FASTAR_ERR_UNSUPPORTED) return rc;
  return launch_hash_simt(dt, x, H, N, D, planes, T, B, codes, st, s);
}

int launch_annca(fastar_dtype dt, const void* q, const void* k_p, const void* v_p,
                 const int32_t* kept_idx, const int32_t* kept_cnt, int H, int F, int n_f, int P,
                 int D, float scale, void* out, void* ws, size_t ws_bytes, int32_t* st, cudaStream_t s) {
  int rc = launch_annca_tc(dt, q, k_p, v_p, kept_idx, kept_cnt, H, F, n_f, P, D, scale, out, ws, ws_bytes,
                           st, s);
  if (rc != FASTAR_ERR_UNSUPPORTED) return rc;
  return launch_annca_simt(dt, q, k_p, v_p, kept_idx, kept_cnt, H, F, n_f, P, D, scale, out, st, s);
}

int launch_annsa(fastar_dtype dt, const void* q, const uint32_t* q_codes, const int32_t* q_perm,
                 const int32_t* q_offsets, int Nq, const fastar_cache* c, float scale, void* out,
                 float* lse, void* ws, int32_t* st, cudaStream_t s) {
  int rc = launch_annsa_tc(dt, q, q_codes, q_perm, q_offsets, Nq, c, scale, out, lse, ws, st, s);
  if (rc != FASTAR_ERR_UNSUPPORTED) return rc;
  return launch_annsa_simt(dt, q, q_codes, Nq, c, scale, out, lse, st, s);
}

size_t annsa_ws_bytes(int H, int Nq, int D, int T) { return annsa_tc_ws_bytes(H, Nq, D, T); }

static bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
static bool dtype_ok(int dt) { return dt == FASTAR_BF16 || dt == FASTAR_F32; }
static bool dim_ok(int D) { return D == 64 || D == 128; }

}  // namespace fastar

using namespace fastar;

extern "C" {

const char* fastar_status_string(int status) {
  switch (status) {
    case FASTAR_OK: return "ok";
    case FASTAR_ERR_ARG: return "invalid argument";
    case FASTAR_ERR_UNSUPPORTED: return "unsupported shape or type";
    case FASTAR_ERR_CUDA: return "CUDA launch error";
    case FASTAR_ERR_WORKSPACE: return "workspace too small";
    case FASTAR_ERR_CAPACITY: return "cache capacity exhausted (device)";
    case FASTAR_ERR_TIMEOUT: return "bounded device wait expired (device)";
    case FASTAR_ERR_DEVICE_ARG: return "out-of-range index found on the device";
    default: return "unknown status";
  }
}

int fastar_version(void) { return 300; }

uint64_t fastar_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int fastar_timing_begin(cudaEvent_t* events, int capacity) {
  if (capacity < 0 || (capacity > 0 && !events)) return FASTAR_ERR_ARG;
  std::lock_guard<std::mutex> lock(g_tmu);
  g_tev = events;
  g_tcap = capacity;
  g_tn = 0;
  g_timing.store(capacity > 0 ? 1 : 0, std::memory_order_release);
  return FASTAR_OK;
}

int fastar_timing_end(void) {
  std::lock_guard<std::mutex> lock(g_tmu);
  g_timing.store(0, std::memory_order_release);
  g_tev = nullptr;
  g_tcap = 0;
  return g_tn;
}

const char* fastar_timing_name(int i) {
  std::lock_guard<std::mutex> lock(g_tmu);
  return (i >= 0 && i < g_tn) ? g_tname[i] : "";
}

size_t fastar_workspace_size(int op, int H, int N, int D, int T, int B, int C) {
  (void)B;
  if (H < 0 || N < 0 || C < 0) return 0;
  switch (op) {
    case FASTAR_OP_MERGE: return merge_ws_bytes(H, N, C);
    case FASTAR_OP_ANNCA: return annca_tc_ws_bytes(H, N, C, D);  // N = frames F, C = prompt tokens P
    case FASTAR_OP_ANNSA: return annsa_ws_bytes(H, N, D, T);
    case FASTAR_OP_ANNSA_PARTS: return annsa_parts_ws_bytes(H, N, D, T);  // T = part_total
    case FASTAR_OP_BRANCH: return branch_ws_bytes(H, T, N, D);  // H = query heads, T = key/value heads
    case FASTAR_OP_QUANT: return quant_ws_bytes(H, N, C, D, T);  // N = Nq, T = bits, C = keys per head
    default: return 0;
  }
}

int fastar_hash(fastar_dtype dt, const void* x, int H, int N, int D, const void* planes, int T,
                int B, uint32_t* codes, int32_t* perm, int32_t* offsets, void* ws, size_t ws_bytes,
                int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_hash");
  (void)ws;
  (void)ws_bytes;
  if (!dtype_ok(dt)) return FASTAR_ERR_UNSUPPORTED;
  if (H < 0 || N < 0 || T < 1 || B < 1 || T > 8) return FASTAR_ERR_ARG;
  if (!dim_ok(D) || T * B > kMaxTB) return FASTAR_ERR_UNSUPPORTED;
  if ((perm == nullptr) != (offsets == nullptr)) return FASTAR_ERR_ARG;
  if (perm && B > kMaxCsrBits) return FASTAR_ERR_UNSUPPORTED;
  if ((size_t)H * N == 0) return FASTAR_OK;
  if (!x || !planes || !codes || !aligned16(x) || !aligned16(planes)) return FASTAR_ERR_ARG;
  int rc = launch_hash(dt, x, H, N, D, planes, T, B, codes, dev_status, stream);
  if (rc != FASTAR_OK || !perm) return rc;
  return launch_csr(codes, H * T, N, nullptr, 1, 1 << B, perm, offsets, dev_status, stream);
}

int fastar_bucket_csr(const uint32_t* codes, int G, int N, int B, int32_t* perm, int32_t* offsets,
                      int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_bucket_csr");
  if (G < 0 || N < 0 || B < 1) return FASTAR_ERR_ARG;
  if (B > kMaxCsrBits) return FASTAR_ERR_UNSUPPORTED;
  if ((size_t)G * N == 0) return FASTAR_OK;
  if (!codes || !perm || !offsets) return FASTAR_ERR_ARG;
  return launch_csr(codes, G, N, nullptr, 1, 1 << B, perm, offsets, dev_status, stream);
}

int fastar_hash_many(fastar_dtype dt, int n_jobs, const fastar_hash_job* jobs, int H, int D,
                     const void* planes, int T, int B, void* ws, size_t ws_bytes, int32_t* dev_status,
                     cudaStream_t stream) {
  CallRange range("fastar_hash_many");
  (void)ws;
  (void)ws_bytes;
  if (!dtype_ok(dt)) return FASTAR_ERR_UNSUPPORTED;
  if (n_jobs < 1 || n_jobs > FASTAR_MAX_HASH_JOBS || !jobs) return FASTAR_ERR_ARG;
  if (H < 0 || T < 1 || B < 1 || T > 8) return FASTAR_ERR_ARG;
  if (!dim_ok(D) || T * B > kMaxTB) return FASTAR_ERR_UNSUPPORTED;
  const void* xs[FASTAR_MAX_HASH_JOBS];
  int Ns[FASTAR_MAX_HASH_JOBS];
  uint32_t* cs[FASTAR_MAX_HASH_JOBS];
  int n = 0;
  for (int j = 0; j < n_jobs; ++j) {
    const fastar_hash_job& q = jobs[j];
    if (q.N < 0 || (q.perm == nullptr) != (q.offsets == nullptr)) return FASTAR_ERR_ARG;
    if (q.perm && B > kMaxCsrBits) return FASTAR_ERR_UNSUPPORTED;
    if ((size_t)H * q.N == 0) continue;
    if (!q.x || !q.codes || !aligned16(q.x)) return FASTAR_ERR_ARG;
    xs[n] = q.x;
    Ns[n] = q.N;
    cs[n] = q.codes;
    ++n;
  }
  if (n == 0) return FASTAR_OK;
  if (!planes || !aligned16(planes)) return FASTAR_ERR_ARG;
  int rc = launch_hash_tc_many(dt, n, xs, Ns, cs, H, D, planes, T, B, dev_status, stream);
  if (rc == FASTAR_ERR_UNSUPPORTED) {
    rc = FASTAR_OK;
    for (int j = 0; j < n && rc == FASTAR_OK; ++j)
      rc = launch_hash(dt, xs[j], H, Ns[j], D, planes, T, B, cs[j], dev_status, stream);
  }
  for (int j = 0; j < n_jobs && rc == FASTAR_OK; ++j) {
    const fastar_hash_job& q = jobs[j];
    if (q.perm && (size_t)H * q.N > 0)
      rc = launch_csr(q.codes, H * T, q.N, nullptr, 1, 1 << B, q.perm, q.offsets, dev_status, stream);
  }
  return rc;
}

static int check_cache(const fastar_cache* c) {
  if (!c) return FASTAR_ERR_ARG;
  if (!dtype_ok(c->dt)) return FASTAR_ERR_UNSUPPORTED;
  if (c->H < 0 || c->C < 1 || c->T < 1 || c->T > 8 || c->B < 1) return FASTAR_ERR_ARG;
  if (!dim_ok(c->D) || c->B > kMaxCsrBits) return FASTAR_ERR_UNSUPPORTED;
  if (!c->K || !c->V || !c->m || !c->codes || !c->last_frame || !c->size || !c->inserted ||
      !c->evicted || !c->perm || !c->offsets)
    return FASTAR_ERR_ARG;
  if (!aligned16(c->K) || !aligned16(c->V)) return FASTAR_ERR_ARG;
  return FASTAR_OK;
}

static int merge_checked(const fastar_cache* cache, const void* k_new, const void* v_new,
                         const uint32_t* codes_new, int F, int n_f, int32_t first_frame, float tau,
                         int32_t* match_out, void* ws, size_t ws_bytes, int32_t* dev_status,
                         cudaStream_t stream, cudaEvent_t codes_ready, int rep = FASTAR_REP_LAST,
                         const void* planes = nullptr, int search = FASTAR_SEARCH_PREV) {
  int rc = check_cache(cache);
  if (rc != FASTAR_OK) return rc;
  if (rep != FASTAR_REP_LAST && rep != FASTAR_REP_MEAN) return FASTAR_ERR_ARG;
  const bool quant_ok = (search & 0xff) == FASTAR_SEARCH_QUANT && (search >> 8) >= 1 && (search >> 8) <= 16;
  if (search != FASTAR_SEARCH_PREV && search != FASTAR_SEARCH_LSH && !quant_ok) return FASTAR_ERR_ARG;
  if (rep == FASTAR_REP_MEAN) {
    if (!planes || !aligned16(planes)) return FASTAR_ERR_ARG;
    if (cache->T * cache->B > 64) return FASTAR_ERR_UNSUPPORTED;
  }
  if (F < 0 || n_f < 0 || n_f > cache->C) return FASTAR_ERR_ARG;
  if (n_f > FASTAR_MAX_FRAME_KEYS) return FASTAR_ERR_UNSUPPORTED;
  if (F == 0 || n_f == 0 || cache->H == 0) {
    // nothing to merge; the caller's stream still follows the event
    if (codes_ready && cudaStreamWaitEvent(stream, codes_ready, 0) != cudaSuccess) {
      (void)cudaGetLastError();
      return FASTAR_ERR_CUDA;
    }
    return FASTAR_OK;
  }
  if (!k_new || !v_new || !codes_new || !aligned16(k_new) || !aligned16(v_new)) return FASTAR_ERR_ARG;
  if (first_frame < 0 || (int64_t)first_frame + F > 0x7fffff00) return FASTAR_ERR_ARG;
  if (tau != tau) return FASTAR_ERR_ARG;
  const size_t need = merge_ws_bytes(cache->H, n_f, cache->C);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  return launch_merge(cache, k_new, v_new, codes_new, F, n_f, first_frame, tau, match_out, ws,
                      dev_status, stream, codes_ready, rep, planes, search);
}

int fastar_tempcache_merge(const fastar_cache* cache, const void* k_new, const void* v_new,
                           const uint32_t* codes_new, int F, int n_f, int32_t first_frame, float tau,
                           int32_t* match_out, void* ws, size_t ws_bytes, int32_t* dev_status,
                           cudaStream_t stream) {
  CallRange range("fastar_tempcache_merge");
  return merge_checked(cache, k_new, v_new, codes_new, F, n_f, first_frame, tau, match_out, ws, ws_bytes,
                       dev_status, stream, nullptr);
}

int fastar_tempcache_merge_ev(const fastar_cache* cache, const void* k_new, const void* v_new,
                              const uint32_t* codes_new, int F, int n_f, int32_t first_frame, float tau,
                              int32_t* match_out, void* ws, size_t ws_bytes, int32_t* dev_status,
                              cudaStream_t stream, cudaEvent_t codes_ready) {
  CallRange range("fastar_tempcache_merge_ev");
  return merge_checked(cache, k_new, v_new, codes_new, F, n_f, first_frame, tau, match_out, ws, ws_bytes,
                       dev_status, stream, codes_ready);
}

int fastar_tempcache_merge_rep(const fastar_cache* cache, const void* k_new, const void* v_new,
                               const uint32_t* codes_new, int F, int n_f, int32_t first_frame, float tau,
                               int rep, const void* planes, int32_t* match_out, void* ws, size_t ws_bytes,
                               int32_t* dev_status, cudaStream_t stream, cudaEvent_t codes_ready) {
  CallRange range("fastar_tempcache_merge_rep");
  return merge_checked(cache, k_new, v_new, codes_new, F, n_f, first_frame, tau, match_out, ws, ws_bytes,
                       dev_status, stream, codes_ready, rep, planes);
}

int fastar_tempcache_merge_search(const fastar_cache* cache, const void* k_new, const void* v_new,
                                  const uint32_t* codes_new, int F, int n_f, int32_t first_frame, float tau,
                                  int search, int32_t* match_out, void* ws, size_t ws_bytes,
                                  int32_t* dev_status, cudaStream_t stream, cudaEvent_t codes_ready) {
  CallRange range("fastar_tempcache_merge_search");
  return merge_checked(cache, k_new, v_new, codes_new, F, n_f, first_frame, tau, match_out, ws, ws_bytes,
                       dev_status, stream, codes_ready, FASTAR_REP_LAST, nullptr, search);
}

int fastar_annca_prune(const uint32_t* q_codes, const uint32_t* p_codes, int H, int F, int n_f,
                       int P, int T, int B, int32_t* kept_idx, int32_t* kept_cnt, void* ws,
                       size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annca_prune");
  (void)ws;
  (void)ws_bytes;
  if (H < 0 || F < 0 || n_f < 0 || P < 0 || T < 1 || T > 8 || B < 1) return FASTAR_ERR_ARG;
  if (B > 16) return FASTAR_ERR_UNSUPPORTED;
  if (H == 0 || F == 0) return FASTAR_OK;
  if (!kept_cnt || (P > 0 && !kept_idx) || (n_f > 0 && !q_codes) || (P > 0 && !p_codes))
    return FASTAR_ERR_ARG;
  return launch_prune(q_codes, p_codes, H, F, n_f, P, T, B, kept_idx, kept_cnt, dev_status, stream);
}

int fastar_annca_attention(fastar_dtype dt, const void* q, const void* k_p, const void* v_p,
                           const int32_t* kept_idx, const int32_t* kept_cnt, int H, int F, int n_f,
                           int P, int D, float scale, void* out, void* ws, size_t ws_bytes,
                           int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annca_attention");
  if (!dtype_ok(dt)) return FASTAR_ERR_UNSUPPORTED;
  if (H < 0 || F < 0 || n_f < 0 || P < 0) return FASTAR_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return FASTAR_ERR_ARG;
  if (!dim_ok(D)) return FASTAR_ERR_UNSUPPORTED;
  if ((size_t)H * F * n_f == 0) return FASTAR_OK;
  if (!q || !out || !kept_cnt || !aligned16(q) || !aligned16(out)) return FASTAR_ERR_ARG;
  if (P > 0 && (!k_p || !v_p || !kept_idx || !aligned16(k_p) || !aligned16(v_p))) return FASTAR_ERR_ARG;
  if (dt == FASTAR_BF16 && D == 128 && P > 0) {
    const size_t need = annca_tc_ws_bytes(H, F, P, D);
    if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  }
  return launch_annca(dt, q, k_p, v_p, kept_idx, kept_cnt, H, F, n_f, P, D, scale, out, ws, ws_bytes,
                      dev_status, stream);
}

int fastar_annsa_attention(fastar_dtype dt, const void* q, const uint32_t* q_codes,
                           const int32_t* q_perm, const int32_t* q_offsets, int Nq,
                           const fastar_cache* cache, float scale, void* out, float* lse, void* ws,
                           size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annsa_attention");
  int rc = check_cache(cache);
  if (rc != FASTAR_OK) return rc;
  if (dt != cache->dt) return FASTAR_ERR_ARG;
  if (Nq < 0) return FASTAR_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return FASTAR_ERR_ARG;
  if (Nq == 0 || cache->H == 0) return FASTAR_OK;
  if (!q || !q_codes || !q_perm || !q_offsets || !out || !aligned16(q) || !aligned16(out))
    return FASTAR_ERR_ARG;
  const size_t need = annsa_ws_bytes(cache->H, Nq, cache->D, cache->T);
  if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return FASTAR_ERR_WORKSPACE;
  return launch_annsa(dt, q, q_codes, q_perm, q_offsets, Nq, cache, scale, out, lse, ws,
                      dev_status, stream);
}

int fastar_annsa_attention_part(fastar_dtype dt, const void* q, const uint32_t* q_codes,
                                const int32_t* q_perm, const int32_t* q_offsets, int Nq,
                                const fastar_cache* cache, float scale, int part_base, int part_total,
                                void* ws, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annsa_attention_part");
  (void)q_offsets;
  int rc = check_cache(cache);
  if (rc != FASTAR_OK) return rc;
  if (dt != cache->dt || Nq < 0) return FASTAR_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return FASTAR_ERR_ARG;
  if (part_total < 1 || part_total > 4 || part_base < 0 || part_base + cache->T > part_total)
    return FASTAR_ERR_ARG;
  if (dt != FASTAR_BF16 || cache->D != 128) return FASTAR_ERR_UNSUPPORTED;
  if (Nq == 0 || cache->H == 0) return FASTAR_OK;
  if (!q || !q_codes || !q_perm || !aligned16(q)) return FASTAR_ERR_ARG;
  const size_t need = annsa_parts_ws_bytes(cache->H, Nq, cache->D, part_total);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  return launch_annsa_parts(q, q_codes, q_perm, Nq, cache, scale, part_base, part_total, ws, dev_status,
                            stream);
}

int fastar_annsa_combine(int H, int Nq, int D, int part_total, const void* ws, size_t ws_bytes, void* out,
                         float* lse, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annsa_combine");
  if (H < 0 || Nq < 0 || part_total < 1 || part_total > 4) return FASTAR_ERR_ARG;
  if (D != 128) return FASTAR_ERR_UNSUPPORTED;
  if (H == 0 || Nq == 0) return FASTAR_OK;
  if (!out || !aligned16(out)) return FASTAR_ERR_ARG;
  const size_t need = annsa_parts_ws_bytes(H, Nq, D, part_total);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  return launch_annsa_combine(H, Nq, part_total, ws, out, lse, dev_status, stream);
}

}  // extern "C"

static int quant_common(int H, int Nq, int N, int D, float scale, int topk, int bits, const void* q,
                        const void* out, void* ws, size_t ws_bytes) {
  if (H < 0 || Nq < 0 || N < 0 || topk < 0) return FASTAR_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return FASTAR_ERR_ARG;
  if (bits < 1 || bits > 16) return FASTAR_ERR_UNSUPPORTED;
  if (D != 128) return FASTAR_ERR_UNSUPPORTED;
  if (H == 0 || Nq == 0) return -1;  // nothing to do
  if (!q || !out || !aligned16(q) || !aligned16(out)) return FASTAR_ERR_ARG;
  if (N == 0) return FASTAR_ERR_ARG;
  const size_t need = quant_ws_bytes(H, Nq, N, D, bits);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  return FASTAR_OK;
}

int fastar_annsa_quant_attention(fastar_dtype dt, const void* q, int Nq, const fastar_cache* cache, float scale,
                                 int topk, int bits, void* out, float* lse, uint32_t* sel_mask, void* ws,
                                 size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annsa_quant_attention");
  int rc = check_cache(cache);
  if (rc != FASTAR_OK) return rc;
  if (dt != cache->dt) return FASTAR_ERR_ARG;
  if (dt != FASTAR_BF16) return FASTAR_ERR_UNSUPPORTED;
  rc = quant_common(cache->H, Nq, cache->C, cache->D, scale, topk, bits, q, out, ws, ws_bytes);
  if (rc == -1) return FASTAR_OK;
  if (rc != FASTAR_OK) return rc;
  return launch_annsa_quant(q, Nq, cache, scale, topk, bits, out, lse, sel_mask, ws, dev_status, stream);
}

int fastar_annca_quant_attention(fastar_dtype dt, const void* q, const void* k_p, const void* v_p, int H, int Nq,
                                 int P, int D, float scale, int topk, int bits, void* out, uint32_t* sel_mask,
                                 void* ws, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_annca_quant_attention");
  if (!dtype_ok(dt)) return FASTAR_ERR_UNSUPPORTED;
  if (dt != FASTAR_BF16) return FASTAR_ERR_UNSUPPORTED;
  int rc = quant_common(H, Nq, P, D, scale, topk, bits, q, out, ws, ws_bytes);
  if (rc == -1) return FASTAR_OK;
  if (rc != FASTAR_OK) return rc;
  if (!k_p || !v_p || !aligned16(k_p) || !aligned16(v_p)) return FASTAR_ERR_ARG;
  return launch_annca_quant(q, k_p, v_p, H, Nq, P, scale, topk, bits, out, sel_mask, ws, dev_status, stream);
}

// ---- branched rollouts

// Rows of a strided tensor start on 16-byte boundaries (a stride counts only
// where there is more than one row along it); rows that are written lie apart.
static bool rows_ok(fastar_dtype dt, const void* x, int64_t head, int64_t token, int H, int N, int D,
                    bool written = false) {
  const int64_t v = dt == FASTAR_BF16 ? 8 : 4;
  if (!x || !aligned16(x)) return false;
  if (H > 1 && (head % v || (written && head < D && head > -D))) return false;
  if (N > 1 && (token % v || (written && token < D && token > -D))) return false;
  return true;
}
static bool plan_ok(const fastar_rope_plan* p, int D) {
  if (!p || p->D != D || p->axes < 1 || p->axes > FASTAR_ROPE_MAX_AXES) return false;
  if (p->pairs < 1 || p->pairs > D / 2 || (p->pairing != FASTAR_PAIRS_ADJACENT && p->pairing != FASTAR_PAIRS_HALVES))
    return false;
  if (p->pairing == FASTAR_PAIRS_HALVES && p->pairs % 8) return false;
  for (int i = 0; i < p->pairs; ++i)
    if (p->axis[i] >= p->axes) return false;
  return true;
}
static int check_pages(const fastar_pages* p) {
  if (!p) return FASTAR_ERR_ARG;
  if (!dtype_ok(p->dt) || !dim_ok(p->D)) return FASTAR_ERR_UNSUPPORTED;
  if (p->H < 1 || p->B < 0 || p->n_pages < 0 || p->max_pages < 0) return FASTAR_ERR_ARG;
  if (p->page < 16 || p->page > 256 || (p->page & (p->page - 1))) return FASTAR_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page > 0x7fffffff) return FASTAR_ERR_UNSUPPORTED;
  if ((int64_t)p->n_pages * p->H > 0x7fffffff / p->page) return FASTAR_ERR_UNSUPPORTED;
  if (p->B > 0 && !p->len) return FASTAR_ERR_ARG;
  if (p->n_pages > 0 && (!p->K || !p->V || !aligned16(p->K) || !aligned16(p->V))) return FASTAR_ERR_ARG;
  if (p->B > 0 && p->max_pages > 0 && (!p->table || p->n_pages == 0)) return FASTAR_ERR_ARG;
  return FASTAR_OK;
}

extern "C" {

int fastar_rope_plan_init(fastar_rope_plan* plan, int D, int axes, const int* dims, int pairing, const double* freq) {
  if (!plan || !dims) return FASTAR_ERR_ARG;
  if (!dim_ok(D)) return FASTAR_ERR_UNSUPPORTED;
  if (axes < 1 || axes > FASTAR_ROPE_MAX_AXES) return FASTAR_ERR_ARG;
  if (pairing != FASTAR_PAIRS_ADJACENT && pairing != FASTAR_PAIRS_HALVES) return FASTAR_ERR_ARG;
  int64_t sum = 0;
  for (int a = 0; a < axes; ++a) {
    if (dims[a] < 0 || dims[a] % 2) return FASTAR_ERR_ARG;
    sum += dims[a];
  }
  if (sum < 2 || sum > D || (pairing == FASTAR_PAIRS_HALVES && sum % 16)) return FASTAR_ERR_ARG;
  for (int i = 0; freq && i < sum / 2; ++i)
    if (!(freq[i] - freq[i] == 0.0)) return FASTAR_ERR_ARG;  // infinite or NaN
  memset(plan, 0, sizeof(*plan));
  plan->D = D;
  plan->axes = axes;
  plan->pairs = (int)(sum / 2);
  plan->pairing = pairing;
  for (int a = 0, p = 0; a < axes; ++a)
    for (int i = 0; i < dims[a] / 2; ++i, ++p) {
      const double f = freq ? freq[p] : pow(10000.0, -2.0 * i / dims[a]);
      const double turns = f / 6.283185307179586476925286766559;
      const double part = turns - floor(turns);  // 1.0 when a tiny negative one is rounded up
      plan->turn[p] = part < 1.0 ? (uint64_t)ldexp(part, 64) : 0u;
      plan->axis[p] = (uint8_t)a;
    }
  return FASTAR_OK;
}

int fastar_rope(fastar_dtype dt, const void* x, int64_t x_head, int64_t x_token, int H, int N, int D,
                const int32_t* pos, const fastar_rope_plan* plan, int inverse, void* out, int64_t out_head,
                int64_t out_token, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_rope");
  if (!dtype_ok(dt) || !dim_ok(D)) return FASTAR_ERR_UNSUPPORTED;
  if (H < 0 || N < 0 || !plan_ok(plan, D)) return FASTAR_ERR_ARG;
  if (H == 0 || N == 0) return FASTAR_OK;
  if (!pos || !rows_ok(dt, x, x_head, x_token, H, N, D) || !rows_ok(dt, out, out_head, out_token, H, N, D, true))
    return FASTAR_ERR_ARG;
  return launch_rope(dt, x, x_head, x_token, H, N, D, pos, plan, inverse, out, out_head, out_token, dev_status, stream);
}

int fastar_page_append(const fastar_pages* pages, const void* k, int64_t k_head, int64_t k_token, const void* v,
                       int64_t v_head, int64_t v_token, int N, const int32_t* cu, const int32_t* pos,
                       const fastar_rope_plan* plan, const void* q, int64_t q_head, int64_t q_token, int Hq,
                       void* q_out, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_page_append");
  int rc = check_pages(pages);
  if (rc != FASTAR_OK) return rc;
  if (N < 0 || Hq < 0 || (plan == nullptr) != (pos == nullptr)) return FASTAR_ERR_ARG;
  if (plan && !plan_ok(plan, pages->D)) return FASTAR_ERR_ARG;
  if (N == 0 || pages->B == 0) return FASTAR_OK;
  if (!cu || !rows_ok(pages->dt, k, k_head, k_token, pages->H, N, pages->D) ||
      !rows_ok(pages->dt, v, v_head, v_token, pages->H, N, pages->D))
    return FASTAR_ERR_ARG;
  if ((q == nullptr) != (Hq == 0) || (q == nullptr) != (q_out == nullptr)) return FASTAR_ERR_ARG;
  if (q && (!rows_ok(pages->dt, q, q_head, q_token, Hq, N, pages->D) || !aligned16(q_out))) return FASTAR_ERR_ARG;
  return launch_page_append(pages, k, k_head, k_token, v, v_head, v_token, N, cu, pos, plan, q, q_head, q_token, Hq,
                            q_out, dev_status, stream);
}

int fastar_branch_attention(fastar_dtype dt, const void* q, int Hq, int N, const int32_t* cu,
                            const fastar_prefix* prefix, const fastar_pages* pages, float scale, int block, void* out,
                            float* lse, void* ws, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  CallRange range("fastar_branch_attention");
  int rc = check_pages(pages);
  if (rc != FASTAR_OK) return rc;
  if (dt != pages->dt || N < 0 || Hq < 0 || Hq % pages->H || block < 0) return FASTAR_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return FASTAR_ERR_ARG;
  if (N == 0 || Hq == 0 || pages->B == 0) return FASTAR_OK;
  if ((int64_t)N * (Hq / pages->H) >= 0x7fffffff - 256) return FASTAR_ERR_UNSUPPORTED;
  if (!q || !cu || !out || !aligned16(q) || !aligned16(out)) return FASTAR_ERR_ARG;
  if (prefix && prefix->C == 0) prefix = nullptr;
  if (prefix) {
    if (prefix->H != pages->H || prefix->D != pages->D || prefix->dt != dt || prefix->C < 0) return FASTAR_ERR_ARG;
    if (!prefix->K || !prefix->V || !aligned16(prefix->K) || !aligned16(prefix->V)) return FASTAR_ERR_ARG;
    if ((int64_t)prefix->H * prefix->C > 0x7fffffff) return FASTAR_ERR_UNSUPPORTED;
  }
  const size_t need = branch_ws_bytes(Hq, pages->H, N, pages->D);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return FASTAR_ERR_WORKSPACE;
  return launch_branch(dt, q, Hq, N, cu, prefix, pages, scale, block, out, lse, ws, dev_status, stream);
}

}  // extern "C"
