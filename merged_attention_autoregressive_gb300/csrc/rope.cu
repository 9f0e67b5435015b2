// Rotary positions with several axes, and the append of new keys and values
// to a paged cache with the rotation applied on the way.
//
// Mathematics.  Pair p of a row turns by the angle pos[axis(p)] * freq(p):
//   y0 = x0 cos - x1 sin,  y1 = x0 sin + x1 cos   (inverse: sin -> -sin).
// The angle is needed modulo one turn only, so the plan holds freq / (2 pi)
// as a 64-bit fixed-point fraction of a turn and the kernel multiplies it by
// the integer position modulo 2^64: no position is too far for it (the error
// of the fraction, 2^-53 from the caller's double, grows to 2^-22 of a turn
// only at |pos| = 2^31), and no 64-bit floating point is used.
//
// What bounds it: memory, one read and one write of every row.  A thread owns
// one token and the two 16-byte vectors of a row that hold whole pairs
// (adjacent pairs: vectors i and i + D/2; halves: a vector and its partner),
// keeps their sines and cosines in registers and walks the heads, so each
// angle is taken once per token and head group, and every access of a warp is
// 64 or 128 contiguous bytes per row on both sides whatever the strides.
// Heads are split over grid y until the grid fills the GPU.  10800 tokens of 40
// bf16 heads: 38.8 us, 5.7 TB/s; appended with their values and queries (18,720
// tokens of 12 heads): 59.3 us, 5.8 TB/s; a few tokens: 4 to 5 us, a launch.
#include <math.h>

#include "common.cuh"

namespace fastar {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // heads in flight per thread: 8 16-byte loads

// One group of heads: rows x[h * xh + n * xt], written to out[h * oh + n * ot]
// (pages: to slot `at` of the token's page).
struct Rows {
  const void* x;
  int64_t xh, xt;
  void* out;
  int64_t oh, ot;
  int H;
};

struct AppendArgs {
  const int32_t* cu;
  const int32_t* len;
  const int32_t* table;
  int B, max_pages, page_shift, n_pages, H;
};

struct RopeArgs {
  Rows q, k, v;           // q: rotated; k: rotated (pages); v: copied (pages)
  const int32_t* pos;     // [N][axes]; null: nothing is rotated
  int N, heads_per_cta;
  uint32_t flip;          // sign bit of the sine for the inverse
};

template <typename T> struct VecInfo { static constexpr int n = 16 / (int)sizeof(T); };

// channels of vector a (0) and b (1) of item i, and the first pair of each;
// pair < 0: copied unturned
template <int V>
__device__ __forceinline__ void item_channels(const fastar_rope_plan& p, int D, int i, int& ca, int& cb) {
  if (p.pairing == FASTAR_PAIRS_HALVES) {
    const int half = p.pairs;  // rotated channels / 2
    if (i * V < half) {
      ca = i * V;
      cb = half + i * V;
    } else {
      ca = 2 * half + (i * V - half) * 2;
      cb = ca + V;
    }
  } else {
    ca = i * V;
    cb = D / 2 + i * V;
  }
}

// N pairs of a row turned by (c, s): (x, y) -> (x c - y s, x s + y c), each in
// fp32 and rounded once to the row's type.
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float a = x, b = y;
  x = a * c - b * s;
  y = a * s + b * c;
}

// Sine and cosine of t / 2^32 of a turn.  32-bit rows: the nearest quarter turn
// is taken off in integers, so that the rest, at most 1/4 half turn, is rounded
// by 2^-27 and not by 2^-25 half turns (the error of an angle is pi times that,
// 2.3e-8); bf16 rows round far above either.
template <typename T>
__device__ __forceinline__ void sincos_turn(uint32_t t, float& s, float& c) {
  constexpr float kStep = 4.656612873077393e-10f;  // 2^-31: half turns
  if constexpr (sizeof(T) == 4) {
    const uint32_t k = (t + 0x20000000u) >> 30;
    float a, b;
    sincospif((float)(int32_t)(t - (k << 30)) * kStep, &a, &b);
    s = __uint_as_float(__float_as_uint(k & 1 ? b : a) ^ (k << 30 & 0x80000000u));
    c = __uint_as_float(__float_as_uint(k & 1 ? a : b) ^ ((k + 1) << 30 & 0x80000000u));
  } else {
    sincospif((float)(int32_t)t * kStep, &s, &c);
  }
}

// Row of position len - back of branch b in the pages of head 0; -1: the position
// is outside the table (as all are of a negative length, whose difference may
// come round to a positive one) or its page outside the pool.
__device__ __forceinline__ int page_row_of(const AppendArgs& ap, int b, int len, int back) {
  const int slot = len - back, pi = slot >> ap.page_shift;
  if (len < 0 || slot < 0 || pi >= ap.max_pages) return -1;
  const int id = ap.table[(size_t)b * ap.max_pages + pi];
  if (id < 0 || id >= ap.n_pages) return -1;
  return ((id * ap.H) << ap.page_shift) + (slot & ((1 << ap.page_shift) - 1));
}

// Whether some token of the call has no place (whole warp, offsets checked): a
// branch per lane, and a page per lane for the pages between its first and last.
__device__ __noinline__ bool some_token_lacks_a_place(const AppendArgs ap) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int b0 = 0; b0 < ap.B; b0 += 32) {
    int len = 0, n = 0;
    if (b0 + lane < ap.B) {
      len = ap.len[b0 + lane];
      n = ap.cu[b0 + lane + 1] - ap.cu[b0 + lane];
    }
    if (n > 0) bad = bad || page_row_of(ap, b0 + lane, len, n) < 0 || page_row_of(ap, b0 + lane, len, 1) < 0;
    for (unsigned more = __ballot_sync(0xffffffffu, n > 1 << ap.page_shift); more; more &= more - 1) {
      const int src = __ffs(more) - 1;
      const int l = __shfl_sync(0xffffffffu, len, src);
      for (int back = __shfl_sync(0xffffffffu, n, src) - (lane << ap.page_shift); back > 0; back -= 32 << ap.page_shift)
        bad = bad || page_row_of(ap, b0 + src, l, back) < 0;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

template <typename T, bool kHalves, bool kAppend>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const __grid_constant__ fastar_rope_plan plan, int D,
                                                        const RopeArgs a, const AppendArgs ap, int32_t* st) {
  constexpr int V = VecInfo<T>::n;     // elements of a 16-byte vector
  pdl_wait();
  const int items = D / (2 * V);       // threads per row
  const int toks = kThreads / items;   // tokens per CTA
  const int tid = threadIdx.x;
  const int lt = tid / items, i = tid % items;
  const int n0 = blockIdx.x * toks, n = n0 + lt;
  const int32_t word = st ? *(volatile const int32_t*)st : 0;
  int page_row = -1;  // row of the token in its page, over all pages of head 0
  bool live = n < a.N;
  if constexpr (kAppend) {
    // the branch of each token of the CTA: every branch marks its own tokens
    __shared__ int s_branch[kThreads / 4], s_first[kThreads / 4], s_count[kThreads / 4];
    for (int t = tid; t < toks; t += kThreads) s_branch[t] = -1;
    __syncthreads();
    bool bad_cu = false;
    for (int b = tid; b < ap.B; b += kThreads) {
      const int lo = ap.cu[b], hi = ap.cu[b + 1];
      if (lo < 0 || hi < lo || hi > a.N || (b == 0 && lo != 0)) {
        bad_cu = true;
        continue;
      }
      for (int t = max(lo, n0); t < min(hi, n0 + toks); ++t) {
        s_branch[t - n0] = b;
        s_first[t - n0] = lo;
        s_count[t - n0] = hi - lo;
      }
    }
    if (bad_cu) status_set(st, FASTAR_ERR_DEVICE_ARG);
    bad_cu = __syncthreads_or(bad_cu) != 0;
    const int b = s_branch[lt];
    live = live && b >= 0;
    if (live) {
      page_row = page_row_of(ap, b, ap.len[b], s_count[lt] - (n - s_first[lt]));
      if (page_row < 0) {
        status_set(st, FASTAR_ERR_DEVICE_ARG);
        live = false;
      }
    }
    if (bad_cu) return;
    // A warp that started before may have set the word, for a token of this very
    // call that has no place: that token alone is skipped.  (The places are
    // looked through only where the word is set; without a barrier, since one in
    // this branch made the whole kernel slower: a chunk 62 us instead of 59.)
    const bool set = __any_sync(0xffffffffu, word != 0);
    if (set && (__any_sync(0xffffffffu, word != 0 && word != FASTAR_ERR_DEVICE_ARG) || !some_token_lacks_a_place(ap))) return;
  } else if (word != 0) {
    return;
  }
  if (!live) return;

  // the item's channels and the sines and cosines of its pairs
  int ca, cb;
  item_channels<V>(plan, D, i, ca, cb);
  constexpr int NP = V;  // pairs per item (V elements in each of two vectors)
  float cs[NP], sn[NP];
  const bool rotated = kHalves ? i * V < plan.pairs : true;
  if (a.pos && rotated) {
    // sines and cosines of the item's pairs (adjacent: V/2 from each vector)
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const int p = kHalves ? ca + e : (e < V / 2 ? ca / 2 + e : cb / 2 + e - V / 2);
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (p < plan.pairs) {
        const int64_t x = a.pos[(size_t)n * plan.axes + plan.axis[p]];
        const uint64_t frac = plan.turn[p] * (uint64_t)x;  // of a turn, modulo 1
        sincos_turn<T>((uint32_t)(frac >> 32), sn[e], cs[e]);
        sn[e] = __uint_as_float(__float_as_uint(sn[e]) ^ a.flip);
      }
    }
  }
  const bool turns = a.pos != nullptr && rotated;

  auto rotate = [&](uint4& u, uint4& w) {
    float x[V], y[V];
    raw_to_float<T, V>(u, x);
    raw_to_float<T, V>(w, y);
    if constexpr (kHalves) {
#pragma unroll
      for (int e = 0; e < V; ++e) turn(x[e], y[e], cs[e], sn[e]);
    } else {
      // channels past the rotated ones are copied (not multiplied by 1 and 0)
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        if (ca / 2 + e < plan.pairs) turn(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
        if (cb / 2 + e < plan.pairs) turn(y[2 * e], y[2 * e + 1], cs[V / 2 + e], sn[V / 2 + e]);
      }
    }
    T* p = reinterpret_cast<T*>(&u);
    T* q = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      Elem<T>::st(p + e, x[e]);
      Elem<T>::st(q + e, y[e]);
    }
  };

  // the heads of this CTA: queries, then keys, then values
  const int total = a.q.H + a.k.H + a.v.H;
  const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, total);
  auto source = [&](int h) -> const T* {
    if (h < a.q.H) return (const T*)a.q.x + h * a.q.xh + n * a.q.xt;
    h -= a.q.H;
    if (h < a.k.H) return (const T*)a.k.x + h * a.k.xh + n * a.k.xt;
    h -= a.k.H;
    return (const T*)a.v.x + h * a.v.xh + n * a.v.xt;
  };
  auto target = [&](int h) -> T* {
    if (h < a.q.H) return (T*)a.q.out + h * a.q.oh + n * a.q.ot;
    h -= a.q.H;
    T* base = (T*)(h < a.k.H ? a.k.out : a.v.out);
    if (h >= a.k.H) h -= a.k.H;
    return base + ((size_t)page_row + ((size_t)h << ap.page_shift)) * D;
  };
  // streaming loads and stores: the rows pass through once (10800 tokens of 40
  // bf16 heads 38.8 us, 61.3 us with plain ones; the append above 59.3 and 88.6 us)
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 u[kUnroll], w[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e)
      if (h + e < h1) {
        const T* s = source(h + e);
        u[e] = __ldcs(reinterpret_cast<const uint4*>(s + ca));
        w[e] = __ldcs(reinterpret_cast<const uint4*>(s + cb));
      }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e)
      if (h + e < h1) {
        if (turns && h + e < a.q.H + a.k.H) rotate(u[e], w[e]);
        T* d = target(h + e);
        __stcs(reinterpret_cast<uint4*>(d + ca), u[e]);
        __stcs(reinterpret_cast<uint4*>(d + cb), w[e]);
      }
  }
  pdl_trigger();
}

template <typename T, bool kAppend>
int launch_rope_t(const fastar_rope_plan& plan, int D, RopeArgs a, const AppendArgs& ap, int32_t* st,
                  cudaStream_t s) {
  const int items = D / (2 * VecInfo<T>::n), toks = kThreads / items;
  const int gx = (a.N + toks - 1) / toks;
  const int total = a.q.H + a.k.H + a.v.H;
  // split the heads until about 32 CTAs per SM are there (the angles are taken
  // again by each part), in steps of the heads in flight: 10800 tokens of 40
  // bf16 heads take 38.8 us so and 45.9 us at twice the parts (the angles).  Half
  // of them is as good: 38.3 us, 4680 tokens 19.4 against 22.9 us, but 20,000
  // tokens 66.2 against 65.3 us and 64.3 against 62.8 us in fp32.
  int parts = (152 * 32 + gx - 1) / gx;
  int per = (total + parts - 1) / parts;
  per = (per + kUnroll - 1) / kUnroll * kUnroll;
  a.heads_per_cta = per;
  const dim3 grid(gx, (total + per - 1) / per);
  cudaError_t rc;
  if (plan.pairing == FASTAR_PAIRS_HALVES)
    rc = launch_pdl(rope_kernel<T, true, kAppend>, grid, dim3(kThreads), 0, s, plan, D, a, ap, st);
  else
    rc = launch_pdl(rope_kernel<T, false, kAppend>, grid, dim3(kThreads), 0, s, plan, D, a, ap, st);
  if (rc != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, kAppend ? "page_append" : "rope");
  return FASTAR_OK;
}

}  // namespace

int launch_rope(fastar_dtype dt, const void* x, int64_t xh, int64_t xt, int H, int N, int D, const int32_t* pos,
                const fastar_rope_plan* plan, int inverse, void* out, int64_t oh, int64_t ot, int32_t* st,
                cudaStream_t s) {
  RopeArgs a = {};
  a.q = {x, xh, xt, out, oh, ot, H};
  a.pos = pos;
  a.N = N;
  a.flip = inverse ? 0x80000000u : 0u;
  const AppendArgs ap = {};
  return dt == FASTAR_BF16 ? launch_rope_t<__nv_bfloat16, false>(*plan, D, a, ap, st, s)
                           : launch_rope_t<float, false>(*plan, D, a, ap, st, s);
}

int launch_page_append(const fastar_pages* pg, const void* k, int64_t kh, int64_t kt, const void* v, int64_t vh,
                       int64_t vt, int N, const int32_t* cu, const int32_t* pos, const fastar_rope_plan* plan,
                       const void* q, int64_t qh, int64_t qt, int Hq, void* q_out, int32_t* st, cudaStream_t s) {
  RopeArgs a = {};
  a.q = {q, qh, qt, q_out, (int64_t)N * pg->D, pg->D, q ? Hq : 0};
  a.k = {k, kh, kt, pg->K, 0, 0, pg->H};
  a.v = {v, vh, vt, pg->V, 0, 0, pg->H};
  a.pos = pos;
  a.N = N;
  AppendArgs ap = {cu, pg->len, pg->table, pg->B, pg->max_pages, 0, pg->n_pages, pg->H};
  while ((1 << ap.page_shift) < pg->page) ++ap.page_shift;
  fastar_rope_plan none = {};
  none.D = pg->D;
  const fastar_rope_plan& p = plan ? *plan : none;
  return pg->dt == FASTAR_BF16 ? launch_rope_t<__nv_bfloat16, true>(p, pg->D, a, ap, st, s)
                               : launch_rope_t<float, true>(p, pg->D, a, ap, st, s);
}

}  // namespace fastar
