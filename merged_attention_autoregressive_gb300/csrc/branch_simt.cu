// fastar_branch_attention on the FP32 pipes.
//
// One CTA of 256 threads takes its run of units (branch.cuh), 64 query rows by
// 64 keys at a time: the scores of a unit (4 x 4 per thread), one pass of
// the running softmax, and the product with the values (4 rows x D/16
// columns per thread, O in registers).  Scores, statistics, probabilities and
// O are fp32; the row statistics of a thread's 4 rows are joined over the 16
// threads of a row by shuffles.  Keys and probabilities share one buffer, so
// two CTAs fit on an SM and one computes while the other waits or takes
// exponentials.  Bound by the FP32 pipes and, where runs are short, by start
// and join: three frames of 256 tokens, 4 heads of 64 channels over 1,536 keys
// take 50 us, of which the multiply-adds are 16 us.
#include <math.h>

#include "branch.cuh"
#include "tc.cuh"

namespace fastar {
namespace {

constexpr int kTM = 64, kTN = 64, kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// (a0, a1) += (x0 y0, x1 y1), one instruction, each as fmaf rounds it.
__device__ __forceinline__ void fma_pair(float& a0, float& a1, float x0, float x1, float y0, float y1) {
  asm("{\n\t.reg .b64 a, x, y;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "fma.rn.f32x2 a, x, y, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error about 2^-22
  return y;
}

// 64 channels leave room for a second stage of keys and values, filled while
// the unit before is computed.
template <int D>
struct SimtSmem {
  static constexpr int kStages = D == 64 ? 2 : 1;
  float Q[kTM][D + 4];
  float K[kStages][kTN][D + 4];  // a stage's keys, then its unit's probabilities [kTM][kTN + 4]
  float V[kStages][kTN][D];
  float bias[kStages][kTN];
  uint64_t full[kStages];
  BranchWalk walk[32];  // of warp 0, a lane each: it lives here between units, out of everybody's registers
  int count, keys_end, full_keys, opens, closes, more;
  BranchUnit next;
  BranchUnit unit[2];  // flag 8: none, the run is over; flag 16: every row sees every one of the 64 keys
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) branch_simt_kernel(BranchArgs a, int32_t* st) {
  branch_touch(a, st);
  pdl_wait();
  extern __shared__ uint4 raw[];
  SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(raw);
  if (block_status_bad(st)) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  constexpr int VN = 4, RV = D / VN;  // vectors per row
  constexpr int kStages = SimtSmem<D>::kStages;
  constexpr int OC = D / 16;                            // O columns per thread
  const float scale2 = a.scale * kLog2e;
  // Warp 0 walks the run and describes unit n, one ahead of its use.
  auto describe = [&](int n) {
    BranchWalk w = sm.walk[tid];
    int count = sm.count, keys_end = sm.keys_end, full_keys = sm.full_keys;
    bool opens = sm.opens, closes = sm.closes, more = sm.more;
    BranchUnit y = sm.next;
    __syncwarp();
    if (more && count == 0) {
      more = w.next(a, y, count, keys_end, opens, closes, n == 0 ? 1 : 0);
      // keys that every row of the item sees: those of its first token, where
      // the item belongs to one branch
      const int r0 = y.t * kTM;
      full_keys = keys_end;
      if (more && y.branch >= 0)
        full_keys = y.lo * a.g <= r0 && (y.lo + y.n) * a.g >= min(r0 + kTM, a.cu[a.B] * a.g)
                        ? branch_limit(r0 / a.g - y.lo, y.n, y.len, a.block)
                        : 0;
    } else if (more) {
      opens = false;
      y.k0 += kTN;
    }
    --count;
    y.nk = max(0, min(kTN, keys_end - y.k0));
    y.flags = !more ? 8
                    : (y.flags & 4) | (opens ? 1 : 0) | (closes && count == 0 ? 2 : 0) |
                          (y.nk == kTN && y.k0 + kTN <= full_keys ? 16 : 0);
    if (more && opens) w.record(a, false);
    if (!more) w.record(a, true);
    sm.walk[tid] = w;
    if (tid == 0) {
      sm.unit[n & 1] = sm.next = y;
      sm.count = count;
      sm.keys_end = keys_end;
      sm.full_keys = full_keys;
      sm.opens = opens;
      sm.closes = closes;
      sm.more = more;
    }
    __syncwarp();
  };
  if (tid < 32) {
    const bool more = sm.walk[tid].start(a, blockIdx.x, st);
    if (tid == 0) {
      sm.count = 0;
      sm.more = more;
      for (int i = 0; i < kStages; ++i) tc::mbar_init(&sm.full[i], 2 * kTN);
      tc::fence_mbar_init();
    }
    __syncwarp();
    describe(0);
    if (more) describe(1);
  }
  const int rows = a.cu[a.B] * a.g;
  float m[4], l[4], o[4][OC];
  bool bad = false;
  // a unit's keys and values, straight into their stage, a row per thread
  // (16-byte copies of all threads took 3800 cycles of a unit to issue, 7 % of 42
  // tokens of 12 heads over 4096 + 1205 keys); its biases
  auto load = [&](int n) {
    const BranchUnit& x = sm.unit[n & 1];
    const int g = kStages == 2 ? n & 1 : 0;
    if (tid < 2 * kTN) {
      const int r = tid % kTN;
      const bool keys = tid < kTN;
      float* const dst = keys ? sm.K[g][r] : sm.V[g][r];
      size_t at = 0;
      bool ok = r < x.nk;
      if (ok && x.branch < 0) {
        at = (size_t)x.h * a.C + x.k0 + r;
      } else if (ok) {
        const int pos = x.k0 + r;
        const int id = a.table[(size_t)x.branch * a.max_pages + (pos >> a.page_shift)];
        ok = id >= 0 && id < a.n_pages;
        at = (((size_t)id * a.H + x.h) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
        bad = bad || !ok;
      }
      if (ok) {
        const float* src = (const float*)(x.branch < 0 ? (keys ? a.pK : a.pV) : (keys ? a.K : a.V)) + at * D;
        tc::mbar_arrive_expect_tx(&sm.full[g], D * 4);
        tc::bulk_load(dst, src, D * 4, &sm.full[g]);
      } else {
        // takes part with weight 0
        for (int c = 0; !keys && c < RV; ++c) *reinterpret_cast<float4*>(dst + c * VN) = make_float4(0.f, 0.f, 0.f, 0.f);
        tc::mbar_arrive(&sm.full[g]);
      }
    } else if (tid < 3 * kTN) {
      const int r = tid - 2 * kTN;
      float b = 0.f;
      if (x.branch < 0 && a.m && r < x.nk) {
        const int c = a.m[(size_t)x.h * a.C + x.k0 + r];
        b = c > 0 ? log2f((float)c) : -INFINITY;
      }
      sm.bias[g][r] = b;
    }
  };
  __syncthreads();
  bool last = sm.unit[0].flags & 8;
  for (int n = 0; !last; ++n) {
    if (n > 0) {
      tc::fence_proxy_async_smem();
      __syncthreads();  // the next unit is described; the products of the one before are done
    }
    const BranchUnit x = sm.unit[n & 1];
    last = sm.unit[(n + 1) & 1].flags & 8;
    const int r0 = x.t * kTM, g = kStages == 2 ? n & 1 : 0;
    if (kStages == 1 || n == 0) load(n);
    if (kStages == 2 && !last) load(n + 1);
    if (x.flags & 1) {
      for (int e = tid; e < kTM * RV; e += kThreads) {
        const int r = e / RV, c = e % RV;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows) {
          const size_t at = (size_t)(x.h * a.g + (int)((r0 + r) % a.g)) * a.N + (size_t)((r0 + r) / a.g);
          v = *reinterpret_cast<const float4*>((const float*)a.q + at * D + c * VN);
        }
        *reinterpret_cast<float4*>(&sm.Q[r][c * VN]) = v;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int d = 0; d < OC; ++d) o[i][d] = 0.f;
      }
    }
    const bool landed = tc::mbar_wait(&sm.full[g], (kStages == 2 ? n >> 1 : n) & 1);
    // a warp computes when one of its 8 rows has keys in the unit
    const int w0 = r0 + (ty & ~1) * 4, lo = x.branch < 0 ? 0 : x.lo * a.g;
    const int hi = x.branch < 0 ? rows : min(rows, (x.lo + x.n) * a.g);
    const bool busy = x.nk > 0 && w0 < hi && w0 + 8 > lo;
    float(*P)[kTN + 4] = reinterpret_cast<float(*)[kTN + 4]>(&sm.K[g][0][0]);
    if (__syncthreads_or(!landed)) {
      if (tid == 0) status_set(st, FASTAR_ERR_TIMEOUT);
      // the copies have landed before the CTA exits
      (void)tc::mbar_wait(&sm.full[g], (kStages == 2 ? n >> 1 : n) & 1);
      if (kStages == 2 && !last) (void)tc::mbar_wait(&sm.full[g ^ 1], ((n + 1) >> 1) & 1);
      break;
    }
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    // two channels at a time: even and odd channels have a sum each
    float s1[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s1[i][j] = 0.f;
    if (busy) {
#pragma unroll 4  // (42 single tokens of 12 heads over 4096 + 1205 keys: 414 us; 8: 423 us; 400 tokens of 8 / 4 heads: 196 us either way)
      for (int k = 0; k < D; k += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&sm.Q[ty * 4 + i][k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&sm.K[g][tx + 16 * j][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fma_pair(s[i][j], s1[i][j], qv[i].x, qv[i].y, kv[j].x, kv[j].y);
            fma_pair(s[i][j], s1[i][j], qv[i].z, qv[i].w, kv[j].z, kv[j].w);
          }
      }
    }
    __syncthreads();  // K has been read: its buffer takes the probabilities
    // a hidden key may hold anything: its values take part with weight 0
    if (x.branch < 0 && a.m && sm.bias[g][tid >> 2] == -INFINITY)
      for (int c = tid & 3; c < RV; c += 4)
        *reinterpret_cast<float4*>(&sm.V[g][tid >> 2][c * VN]) = make_float4(0.f, 0.f, 0.f, 0.f);
    int sees = 0;  // rows that see a key of the unit, or are nobody's
    if (busy) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty * 4 + i;
        const int seen = x.flags & 16 ? kTN : r < rows ? branch_row_keys(a, x, r) : 0;
        sees |= (seen > 0 || r >= rows ? 1 : 0) << i;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = tx + 16 * j;
          const float bias = sm.bias[g][c];
          s[i][j] = c < seen && bias != -INFINITY ? fmaf(s[i][j] + s1[i][j], scale2, bias) : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m[i], top);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = ex2(s[i][j] - base);
          sum += p;
          P[ty * 4 + i][tx + 16 * j] = p;
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        m[i] = mn;
        l[i] = l[i] * alpha + sum;
#pragma unroll
        for (int d = 0; d < OC; ++d) o[i][d] *= alpha;
      }
    }
    __syncthreads();
    if (tid < 32 && !last) describe(n + 2);  // in the place of this unit, of which everybody has a copy
    if (sees == 15) {
#pragma unroll 2
      for (int k = 0; k < kTN; k += 4) {
        float4 pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4*>(&P[ty * 4 + i][k]);
#pragma unroll
        for (int c = 0; c < OC / 4; ++c) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.V[g][k + kk][tx * 4 + 64 * c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
              fma_pair(o[i][4 * c], o[i][4 * c + 1], p, p, v.x, v.y);
              fma_pair(o[i][4 * c + 2], o[i][4 * c + 3], p, p, v.z, v.w);
            }
          }
        }
      }
    } else if (sees) {
      // a unit of another branch leaves a row as it is, also where its values
      // are no numbers (a weight of 0 would not)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sees >> i & 1) {
#pragma unroll 2
          for (int k = 0; k < kTN; k += 4) {
            const float4 pv = *reinterpret_cast<const float4*>(&P[ty * 4 + i][k]);
#pragma unroll
            for (int c = 0; c < OC / 4; ++c) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const float4 v = *reinterpret_cast<const float4*>(&sm.V[g][k + kk][tx * 4 + 64 * c]);
                const float p = kk == 0 ? pv.x : kk == 1 ? pv.y : kk == 2 ? pv.z : pv.w;
                fma_pair(o[i][4 * c], o[i][4 * c + 1], p, p, v.x, v.y);
                fma_pair(o[i][4 * c + 2], o[i][4 * c + 3], p, p, v.z, v.w);
              }
            }
          }
        }
    }
    if (x.flags & 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int lr = ty * 4 + i;
        const int r = r0 + lr;
        if (r >= rows) continue;
        if (x.flags & 4) {
          const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // a NaN sum stays one
          const size_t at = (size_t)(x.h * a.g + (int)(r % a.g)) * a.N + (size_t)(r / a.g);
#pragma unroll
          for (int c = 0; c < OC / 4; ++c) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = o[i][4 * c + e] * inv;
            st_vec<float, 4>((float*)a.out + at * D + tx * 4 + 64 * c, v);
          }
          if (a.lse && tx == 0) a.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
        } else {
          const size_t at = (size_t)x.slot * a.slot_rows + lr;
#pragma unroll
          for (int c = 0; c < OC / 4; ++c)
            st_vec<float, 4>(a.po + ((size_t)x.slot * D + 4 * (tx + 16 * c)) * a.slot_rows + 4 * lr, &o[i][4 * c]);
          if (tx == 0) a.pml[at] = make_float2(m[i], l[i]);
        }
      }
    }
  }
  if (bad) status_set(st, FASTAR_ERR_DEVICE_ARG);
  pdl_trigger();
}

template <int D>
int launch_t(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  constexpr int smem = (int)sizeof(SimtSmem<D>);
  auto kernel = branch_simt_kernel<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      launch_pdl(kernel, dim3(a.G), dim3(kThreads), smem, s, a, st) != cudaSuccess) {
    (void)cudaGetLastError();
    return FASTAR_ERR_CUDA;
  }
  FASTAR_LAUNCHED(s, "branch_simt");
  return FASTAR_OK;
}

}  // namespace

int launch_branch_simt(const BranchArgs& a, int32_t* st, cudaStream_t s) {
  return a.D == 128 ? launch_t<128>(a, st, s) : launch_t<64>(a, st, s);
}

}  // namespace fastar
