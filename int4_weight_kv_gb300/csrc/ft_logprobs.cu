// Log probabilities of given tokens, with the distribution's entropy, the token's
// rank and the k most probable alternatives.
//
//   m = max x, z = sum 2^((x - m) log2 e):  log z + m is the normaliser,
//   entropy = log z - sum e (x - m) / z.
//
// A cluster of CTAs per row, each streaming a slice once with 16-byte loads, the next
// round's in flight while one is used: running maximum, sum and weighted sum per thread
// (a moved maximum rescales them), and the target's rank counted by comparison.  The
// alternatives cost the stream nothing: with t the k-th largest of the 256 threads'
// maxima, only elements >= t can be among the k largest, and only the threads whose
// maximum reaches t (k of them, more with ties) hold such elements.  The CTA reads those
// threads' vectors once more, lists what reaches t, and ranks the list.  (Filtering every
// round through a running threshold instead cost 36 us of 213 for k = 1 and 53 of 88 for
// k = 20, 256 rows of 128256.)
// CTA 0 joins the slices through distributed shared memory: one launch, no workspace.
// Bound by HBM for many rows (2048 FP32 rows of 128256, k = 1: 192 us, 5.5 TB/s); a single row by its
// latency, hence up to 8 CTAs for it (9.2 us, k = 5).
//
// Alternatives are ordered by a 64-bit key (the value as an ordered integer, then the
// lower index), so ties have one answer whatever order the row is read in.
#include <algorithm>

#include "ft_internal.cuh"

namespace ft {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32, kLpMaxTop = 32, kLpMaxCluster = 8;
constexpr int kLpElems = 16;                              // elements of one thread in one round
constexpr int kLpKeep = 256;                              // listed alternatives before a cut
constexpr int kLpScan = 8;                                // elements a thread reads again in one round
constexpr int kLpList = kLpThreads * kLpScan + kLpKeep;   // all of a round may pass
constexpr float kLog2e = 1.44269504088896341f;

struct LogprobParams {
  const void* x;
  int64_t stride;
  const int32_t* target;
  float *logprob, *entropy, *top_val;
  int32_t *rank, *top_id, *status;
  int V, top;
};

typedef unsigned long long lp_key_t;

__device__ __forceinline__ uint32_t lp_order(float v) {  // -0 = +0
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Larger key: larger value, then lower index.
__device__ __forceinline__ lp_key_t lp_key(float v, int i) { return ((lp_key_t)lp_order(v) << 32) | (uint32_t)~i; }
__device__ __forceinline__ float lp_key_value(lp_key_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Running statistics: maximum m, z = sum e^d, u = sum e^d d, d = x - m (m itself is not scaled by
// log2 e, which would overflow for logits near FP32's largest).
struct LpStat {
  float m, z, u;
  __device__ __forceinline__ void move(float to) {  // to >= m
    if (m == -INFINITY) {
      m = to;  // z = u = 0
    } else if (to != m) {
      const float f = lp_ex2((m - to) * kLog2e);
      u = f == 0.0f ? 0.0f : f * fmaf(m - to, z, u);
      z *= f;
      m = to;
    }
  }
  __device__ __forceinline__ void join(LpStat o) {
    const float to = fmaxf(m, o.m);
    move(to);
    o.move(to);
    z += o.z;
    u += o.u;
  }
};

struct LpShared {
  lp_key_t list[kLpList];
  lp_key_t best[kLpMaxTop];
  lp_key_t inbox[kLpMaxCluster * kLpMaxTop];  // CTA 0: the slices' best
  lp_key_t high[kLpThreads];
  float4 stat[kLpMaxCluster];                 // CTA 0: the slices' (m, z, u, rank)
  float4 wstat[kLpWarps];
  __align__(16) float top[kLpThreads];        // the threads' maxima
  uint8_t cand[kLpThreads];
  uint32_t tau;
  lp_key_t tau_key;
  int count, n_cand;
};

// The k largest of n <= 2 kLpThreads keys (0: none), in order, to out; all threads of the CTA.
__device__ __forceinline__ void lp_merge(const lp_key_t* list, lp_key_t* out, int n, int k) {
  const int tid = threadIdx.x;
  const lp_key_t a = tid < n ? list[tid] : 0, b = tid + kLpThreads < n ? list[tid + kLpThreads] : 0;
  int before_a = 0, before_b = 0;
  if (tid < k) out[tid] = 0;
  __syncthreads();
#pragma unroll 8
  for (int j = 0; j < n; ++j) {
    const lp_key_t o = list[j];
    before_a += o > a;
    before_b += o > b;
  }
  if (a && before_a < k) out[before_a] = a;
  if (b && before_b < k) out[before_b] = b;
  __syncthreads();
}
static_assert(kLpMaxCluster * kLpMaxTop <= 2 * kLpThreads, "lp_merge");

// The list's k largest, in order, to best.  A longer list than lp_merge takes is first cut the
// way the row is: the k-th largest of the threads' maxima bounds what can matter.
__device__ __forceinline__ void lp_rank(LpShared& s, int k) {
  const int tid = threadIdx.x;
  int n = s.count;
  while (n > 2 * kLpThreads) {  // leaves at most k ceil(n / kLpThreads) keys, under half of them
    lp_key_t mine = 0;
    for (int i = tid; i < n; i += kLpThreads) mine = max(mine, s.list[i]);
    s.high[tid] = mine;
    __syncthreads();
    int before = 0;
    for (int j = 0; j < kLpThreads; ++j) before += s.high[j] > mine;
    if (before == k - 1) s.tau_key = mine;
    if (tid == 0) s.count = 0;
    __syncthreads();
    const lp_key_t t = s.tau_key;
    lp_key_t held[(kLpList + kLpThreads - 1) / kLpThreads];
#pragma unroll
    for (int q = 0; q < (kLpList + kLpThreads - 1) / kLpThreads; ++q) {
      const int i = q * kLpThreads + tid;
      held[q] = i < n ? s.list[i] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < (kLpList + kLpThreads - 1) / kLpThreads; ++q)
      if (held[q] >= t && held[q]) s.list[atomicAdd(&s.count, 1)] = held[q];
    __syncthreads();
    n = s.count;
  }
  lp_merge(s.list, s.best, n, k);
}

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const LogprobParams p) {
  constexpr int E = BF16 ? 8 : 4, U = kLpElems / E;  // elements of a 16-byte vector, vectors of a thread's round
  constexpr int kStep = U * kLpThreads;              // vectors of the CTA's round
  griddep_serve();
  extern __shared__ __align__(16) uint8_t lp_smem[];
  LpShared& s = *reinterpret_cast<LpShared*>(lp_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = p.V, top = p.top;
  uint32_t rank_in, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_in));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int64_t row = blockIdx.x / ctas;
  if (ctas > 1) cluster_arrive();  // paired with the wait before the first store to CTA 0
  const uint8_t* base = static_cast<const uint8_t*>(p.x) + row * p.stride * (BF16 ? 2 : 4);
  auto at = [&](int i) {
    return BF16 ? bf16_bits_to_f32(__ldcg(reinterpret_cast<const uint16_t*>(base) + i))
                : __ldcg(reinterpret_cast<const float*>(base) + i);
  };
  const int t = p.target ? __ldcg(p.target + row) : -1;
  const bool has = t >= 0 && t < V;
  const float xt = has ? at(t) : INFINITY;  // without a target nothing is before it
  // vector v holds elements v E - lead .. + E - 1, 16-byte aligned; the first and the last may be partial
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / (BF16 ? 2 : 4));
  const uint8_t* vec0 = base - lead * (BF16 ? 2 : 4);
  const int nvec = (lead + V + E - 1) / E;
  const int v0 = (int)((int64_t)nvec * rank_in / ctas), v1 = (int)((int64_t)nvec * (rank_in + 1) / ctas);
  float run_m = -INFINITY;                      // this thread's statistics, the sums in pairs
  f32x2 run_z(0.0f, 0.0f), run_u(0.0f, 0.0f);
  int above = 0;
  // 16-byte vectors, or their elements inside the row at its ends; the others -infinity
  auto fetch = [&](int r, uint4 (&q)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = r + i * kLpThreads + tid;
      const int e0 = v * E - lead;
      if (r > 0 && r + U * kLpThreads < v1) {  // a round inside the row and the slice
        q[i] = __ldcg(reinterpret_cast<const uint4*>(vec0) + v);
      } else if (v < v1 && e0 >= 0 && e0 + E <= V) {
        q[i] = __ldcg(reinterpret_cast<const uint4*>(vec0) + v);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = BF16 ? 0xFF80FF80u : 0xFF800000u;
        if (v < v1) {
#pragma unroll
          for (int k = 0; k < E; ++k) {
            if (e0 + k < 0 || e0 + k >= V) continue;
            if (BF16) {
              const uint32_t h = __ldcg(reinterpret_cast<const uint16_t*>(base) + e0 + k);
              w[k / 2] = (k & 1) ? (w[k / 2] & 0xFFFFu) | (h << 16) : (w[k / 2] & 0xFFFF0000u) | h;
            } else {
              w[k % 4] = __ldcg(reinterpret_cast<const uint32_t*>(base) + e0 + k);
            }
          }
        }
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto use = [&](int r, const uint4 (&q)[U]) {
    float x[kLpElems];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int k = 0; k < E; ++k)
        x[i * E + k] = BF16 ? __uint_as_float((k & 1) ? (w[k / 2] & 0xFFFF0000u) : (w[k / 2] << 16))
                            : __uint_as_float(w[k % 4]);
    }
    float bm = x[0];
#pragma unroll
    for (int k = 1; k < kLpElems; ++k) bm = fmaxf(bm, x[k]);
    if (bm > run_m) {
      const float f = run_m == -INFINITY ? 0.0f : lp_ex2((run_m - bm) * kLog2e);
      const float d = f == 0.0f ? 0.0f : run_m - bm;
      const f32x2 f2(f, f);
      run_u = mul2(f2, fma2(f32x2(d, d), run_z, run_u));
      run_z = mul2(f2, run_z);
      run_m = bm;
    }
    const float m = run_m == -INFINITY ? 0.0f : run_m;
    const f32x2 m2(-m, -m), l2(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < kLpElems; k += 2) {
      const f32x2 d2 = add2(f32x2(x[k], x[k + 1]), m2);
      float d0, d1, s0, s1;
      mul2(d2, l2).get(s0, s1);
      d2.get(d0, d1);
      const f32x2 e2(lp_ex2(s0), lp_ex2(s1));
      run_z = add2(run_z, e2);                                                // a NaN or +infinity stays in z
      run_u = fma2(e2, f32x2(fmaxf(d0, -1000.0f), fmaxf(d1, -1000.0f)), run_u);  // 0 x -infinity of a masked logit is 0
    }
    if (bm >= xt) {  // without a target xt is +infinity: a row that reaches it has no rank anyway
      const int lo = r * E - lead;
      if (r > 0 && r + kStep < v1 && (lo > t || lo + kStep * E <= t)) {  // all of the round behind the target, or before it
        if (lo > t) {
#pragma unroll
          for (int k = 0; k < kLpElems; ++k) above += x[k] > xt;
        } else {
#pragma unroll
          for (int k = 0; k < kLpElems; ++k) above += x[k] >= xt;
        }
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int v = r + i * kLpThreads + tid, e0 = v * E - lead;
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float y = x[i * E + k];
            above += (y > xt || (y == xt && e0 + k < t)) && e0 + k >= 0 && v < v1;
          }
        }
      }
    }
  };

  uint4 cur[U], nxt[U];
  fetch(v0, cur);
  for (int r = v0; r < v1; r += kStep) {
    if (r + kStep < v1) fetch(r + kStep, nxt);
    use(r, cur);
#pragma unroll
    for (int i = 0; i < U; ++i) cur[i] = nxt[i];
  }
  if (top > 0) {
    s.top[tid] = run_m;
    if (tid == 0) s.count = s.n_cand = 0, s.tau = 0xFFFFFFFFu, s.tau_key = 0;
    __syncthreads();
    int before = 0;
#pragma unroll 4
    for (int i = 0; i < kLpThreads; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(s.top + i);
      before += (f.x > run_m) + (f.y > run_m) + (f.z > run_m) + (f.w > run_m);
    }
    if (before < top) atomicMin(&s.tau, lp_order(run_m));  // the lowest of the k largest maxima
    __syncthreads();
    const uint32_t tau_o = s.tau;
    const float tau = lp_key_value((lp_key_t)tau_o << 32);
    if (run_m >= tau) s.cand[atomicAdd(&s.n_cand, 1)] = (uint8_t)tid;  // order does not matter
    __syncthreads();
    // the candidates' vectors again: item w is vector w % nv of thread cand[w / nv]
    const int nv = (v1 - v0 + kLpThreads - 1) / kLpThreads, items = s.n_cand * nv;
    constexpr int kPer = kLpScan / E;
    lp_key_t floor_key = 0;  // once cut, keys must be above the k-th best
    for (int w0 = 0; w0 < items; w0 += kPer * kLpThreads) {
      bool full = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int w = w0 + i * kLpThreads + tid;
        if (w < items) {
          const int c = w / nv, v = v0 + (w - c * nv) * kLpThreads + s.cand[c], e0 = v * E - lead;
          if (v < v1) {
            const bool inside = e0 >= 0 && e0 + E <= V;
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (inside) q = __ldcg(reinterpret_cast<const uint4*>(vec0) + v);
            const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < E; ++k) {
              if (!inside && (e0 + k < 0 || e0 + k >= V)) continue;
              const float x = !inside ? at(e0 + k)
                              : BF16  ? __uint_as_float((k & 1) ? (wd[k / 2] & 0xFFFF0000u) : (wd[k / 2] << 16))
                                      : __uint_as_float(wd[k % 4]);
              if (x >= tau) {
                const lp_key_t key = lp_key(x, e0 + k);
                if (key > floor_key) {
                  const int n = atomicAdd(&s.count, 1);
                  s.list[n] = key;
                  full |= n >= kLpKeep;
                }
              }
            }
          }
        }
      }
      if (__syncthreads_or(full) && w0 + kPer * kLpThreads < items) {
        lp_rank(s, top);
        floor_key = s.best[top - 1];
        if (tid < top) s.list[tid] = s.best[tid];
        if (tid == 0) s.count = top;
        __syncthreads();
      }
    }
    lp_rank(s, top);
  }

  // ---- the CTA's statistics, in warp order
  LpStat st;
  {
    float a, b;
    st.m = run_m;
    run_z.get(a, b);
    st.z = a + b;
    run_u.get(a, b);
    st.u = a + b;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LpStat b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.z = __shfl_xor_sync(0xffffffffu, st.z, o);
    b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
    st.join(b);
    above += __shfl_xor_sync(0xffffffffu, above, o);
  }
  if (lane == 0) s.wstat[warp] = make_float4(st.m, st.z, st.u, __int_as_float(above));
  __syncthreads();
  if (ctas > 1) cluster_wait();
  if (tid == 0) {
    LpStat all = {-INFINITY, 0.0f, 0.0f};
    int cnt = 0;
    for (int w = 0; w < kLpWarps; ++w) {
      const float4 q = s.wstat[w];
      LpStat b = {q.x, q.y, q.z};
      all.join(b);
      cnt += __float_as_int(q.w);
    }
    const float4 q = make_float4(all.m, all.z, all.u, __int_as_float(cnt));
    uint32_t dst;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&s.stat[rank_in])));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(q.x), "f"(q.y), "f"(q.z), "f"(q.w)
                 : "memory");
  }
  if (tid < top) {
    uint32_t dst;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&s.inbox[rank_in * top + tid])));
    const lp_key_t key = s.best[tid];
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst), "l"(key) : "memory");
  }
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (rank_in != 0) return;

  // ---- CTA 0: the slices joined in order
  LpStat all = {-INFINITY, 0.0f, 0.0f};
  int cnt = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const float4 q = s.stat[c];
    LpStat b = {q.x, q.y, q.z};
    all.join(b);
    cnt += __float_as_int(q.w);
  }
  const bool bad = !(all.z > 0.0f && all.z < INFINITY);  // a NaN or +infinity, or nothing that is possible
  const float lz = logf(all.z), mx = all.m, nanv = __int_as_float(0x7FC00000);
  auto logp = [&](float v) { return (v - mx) - lz; };
  if (tid == 0) {
    if (bad || (t != -1 && !has)) set_status(p.status, FT_DEV_RANGE);
    if (p.logprob) p.logprob[row] = t == -1 ? 0.0f : (bad || !has) ? nanv : logp(xt);
    if (p.entropy) p.entropy[row] = bad ? nanv : lz - all.u / all.z;
    if (p.rank) p.rank[row] = (bad || !has) ? -1 : cnt;
  }
  if (top > 0) {
    if (ctas > 1) lp_merge(s.inbox, s.best, (int)ctas * top, top);
    if (tid < top) {
      const lp_key_t key = s.best[tid];
      p.top_id[row * top + tid] = bad ? -1 : (int)~(uint32_t)key;
      p.top_val[row * top + tid] = bad ? nanv : logp(lp_key_value(key));
    }
  }
}

// CTAs per row: as many as keep the grid within one and a half CTAs a SM, with two rounds
// each.  Every further CTA pays the alternatives' fixed cost again.  Measured (FP32, V = 128256,
// k = 1; us): one row 16.7 / 12.9 / 10.4 / 9.2 / 8.8 for 1 / 2 / 4 / 8 / 16 CTAs, 32 rows 17.0 / 12.8
// / 10.7 / 11.3 / 18.3, 256 rows 33 / 41 / 44 / 58 / 108.
static int lp_cluster(int N, int V) {
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  const int rounds = (V + kLpThreads * kLpElems - 1) / (kLpThreads * kLpElems);
  int c = 1;
  while (c < kLpMaxCluster && 4 * c <= rounds && (int64_t)N * 4 * c <= (int64_t)3 * sms) c *= 2;
  return c;
}

template <bool BF16>
static cudaError_t launch_logprobs(const LogprobParams& p, int N, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(LpShared));
    if (e != cudaSuccess) return e;
    allowed[dev] = 1;
  }
  const int ctas = lp_cluster(N, p.V);
  return launch_served(logprobs_kernel<BF16>, dim3((unsigned)((int64_t)N * ctas)), dim3(kLpThreads), sizeof(LpShared), st, ctas, p);
}

}  // namespace ft

extern "C" {

int ft_logprobs(const void* logits, int dtype, int64_t row_stride, int N, int V, const int32_t* targets, int top_k,
                float* logprob, float* entropy, int32_t* rank, int32_t* top_ids, float* top_logprobs,
                int32_t* dev_status, ft_stream stream) {
  if (dtype != FT_BF16 && dtype != FT_F32) return FT_ERR_INVALID_ARG;
  if (N < 0 || V < 1 || top_k < 0 || row_stride < V) return FT_ERR_INVALID_ARG;
  if (top_k > ft::kLpMaxTop || top_k > V || V > (1 << 30)) return FT_ERR_UNSUPPORTED;
  if (N == 0) return FT_OK;
  if (!logits || (top_k > 0 && (!top_ids || !top_logprobs)) || ((logprob || rank) && !targets)) return FT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == FT_F32 ? 4 : 2)) return FT_ERR_INVALID_ARG;
  ft::LogprobParams p = {};
  p.x = logits;
  p.stride = row_stride;
  p.target = targets;
  p.logprob = logprob;
  p.entropy = entropy;
  p.rank = rank;
  p.top_id = top_ids;
  p.top_val = top_logprobs;
  p.status = dev_status;
  p.V = V;
  p.top = top_k;
  const cudaError_t e = dtype == FT_BF16 ? ft::launch_logprobs<true>(p, N, (cudaStream_t)stream)
                                         : ft::launch_logprobs<false>(p, N, (cudaStream_t)stream);
  return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
