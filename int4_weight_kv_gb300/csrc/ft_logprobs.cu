// Log probabilities of given tokens, with the distribution's entropy, the token's
// rank and the k most probable alternatives.
//
//   m = max x, z = sum 2^((x - m) log2 e):  log z + m is the normaliser,
//   entropy = log z - sum e (x - m) / z.
//
// A cluster of CTAs per row, each streaming a slice once with 16-byte loads, the next
// round's in flight while one is used: running maximum, sum and weighted sum per thread
// (a moved maximum rescales them), the target's rank counted by comparison, and the
// alternatives filtered through a threshold: only elements above the k-th best so far
// reach the warp's list, which is cut back to k when it passes kLpKeep.  The first
// threshold is the k-th largest of the lanes' first maxima, so few elements pass even
// then; the best threshold of any warp serves all of the CTA.  Warps meet only at the
// end: a barrier in every round cost a third of the time.
// CTA 0 joins the slices through distributed shared memory: one launch, no workspace.
// Bound by HBM for many rows; a single row by its latency, hence up to 16 CTAs for it.
//
// Alternatives are ordered by a 64-bit key (the value as an ordered integer, then the
// lower index), so ties have one answer whatever order the row is read in.
#include <algorithm>

#include "ft_internal.cuh"

namespace ft {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32, kLpMaxTop = 32, kLpMaxCluster = 16;
constexpr int kLpElems = 16;                              // elements of one thread in one round
constexpr int kLpKeep = 2 * kLpMaxTop + 4;                // listed alternatives of a warp before a cut, at most
constexpr int kLpList = 32 * kLpElems + kLpKeep;          // all of a warp's round may pass
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

// Pairs of FP32 values: one instruction for two elements.
struct lp2 {
  unsigned long long v;
  __device__ __forceinline__ lp2() {}
  __device__ __forceinline__ lp2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ lp2 add2(lp2 a, lp2 b) {
  lp2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ lp2 mul2(lp2 a, lp2 b) {
  lp2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ lp2 fma2(lp2 a, lp2 b, lp2 c) {
  lp2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
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
  lp_key_t list[kLpWarps][kLpList];
  lp_key_t cut[kLpWarps][kLpMaxTop];          // scratch
  lp_key_t best[kLpWarps * kLpMaxTop];        // each warp's best, then the CTA's
  lp_key_t inbox[kLpMaxCluster * kLpMaxTop];  // CTA 0: the slices' best
  float4 stat[kLpMaxCluster];                 // CTA 0: the slices' (m, z, u, rank)
  float4 wstat[kLpWarps];
  uint32_t tau;                               // largest threshold of any warp (lp_order)
};

// The k-th largest of one value per lane (the lowest where fewer lanes hold one).
template <typename T>
__device__ __forceinline__ T lp_kth(T mine, int k) {
  const int lane = threadIdx.x & 31;
  int before = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const T o = __shfl_sync(0xffffffffu, mine, i);
    before += o > mine || (o == mine && i < lane);
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, before == k - 1)) - 1;
  return __shfl_sync(0xffffffffu, mine, max(src, 0));
}

// Cuts a warp's list of n keys to its k largest, in order, at the front of the list; returns how many.
// `out` is scratch of k keys.
__device__ __noinline__ int lp_cut(lp_key_t* list, lp_key_t* out, int n, int k) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (n > 4 * kLpMaxTop) {
    // the k-th largest of the lanes' maxima bounds the k-th largest from below, and only the
    // k lanes at or above it hold keys that pass: at most k n / 32 are left
    lp_key_t mx = 0;
    for (int i = lane; i < n; i += 32) mx = max(mx, list[i]);
    const lp_key_t t = lp_kth(mx, k);
    int kept = 0;
    for (int i = lane; i - lane < n; i += 32) {
      const lp_key_t key = i < n ? list[i] : 0;
      const bool in = i < n && key >= t;
      const uint32_t votes = __ballot_sync(0xffffffffu, in);  // every lane has read its key
      if (in) list[kept + __popc(votes & ((1u << lane) - 1))] = key;
      kept += __popc(votes);
      __syncwarp();
    }
    n = kept;
  }
  for (int i0 = 0; i0 < n; i0 += 128) {  // every key's place among the others, four keys a lane
    lp_key_t mine[4];
    int before[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) mine[q] = i0 + 32 * q + lane < n ? list[i0 + 32 * q + lane] : ~0ull;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const lp_key_t o = list[j];
#pragma unroll
      for (int q = 0; q < 4; ++q) before[q] += o > mine[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i0 + 32 * q + lane < n && before[q] < k) out[before[q]] = mine[q];
  }
  __syncwarp();
  if (lane < min(n, k)) list[lane] = out[lane];
  __syncwarp();
  return min(n, k);
}

// The k largest of n <= 2 kLpThreads keys (0: none), in order, to out; all threads of the CTA.
__device__ __forceinline__ void lp_merge(const lp_key_t* list, lp_key_t* out, int n, int k) {
  const int tid = threadIdx.x;
  const lp_key_t a = tid < n ? list[tid] : 0, b = tid + kLpThreads < n ? list[tid + kLpThreads] : 0;
  int before_a = 0, before_b = 0;
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
static_assert(kLpMaxCluster * kLpMaxTop <= 2 * kLpThreads && kLpWarps * kLpMaxTop <= 2 * kLpThreads, "lp_merge");

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const LogprobParams p) {
  constexpr int E = BF16 ? 8 : 4, U = kLpElems / E;  // elements of a 16-byte vector, vectors of a thread's round
  constexpr int kStep = U * kLpThreads;              // vectors of the CTA's round
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
    return BF16 ? bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(base) + i))
                : __ldg(reinterpret_cast<const float*>(base) + i);
  };
  const int t = p.target ? p.target[row] : -1;
  const bool has = t >= 0 && t < V;
  const float xt = has ? at(t) : INFINITY;  // without a target nothing is before it
  // vector v holds elements v E - lead .. + E - 1, 16-byte aligned; the first and the last may be partial
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / (BF16 ? 2 : 4));
  const uint8_t* vec0 = base - lead * (BF16 ? 2 : 4);
  const int nvec = (lead + V + E - 1) / E;
  const int v0 = (int)((int64_t)nvec * rank_in / ctas), v1 = (int)((int64_t)nvec * (rank_in + 1) / ctas);
  float run_m = -INFINITY;                      // this thread's statistics, the sums in pairs
  lp2 run_z(0.0f, 0.0f), run_u(0.0f, 0.0f);
  int above = 0;
  if (tid == 0) s.tau = 0;
  __syncthreads();

  // 16-byte vectors, or their elements inside the row at its ends; the others -infinity
  auto fetch = [&](int r, uint4 (&q)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = r + i * kLpThreads + tid;
      const int e0 = v * E - lead;
      if (r > 0 && r + U * kLpThreads < v1) {  // a round inside the row and the slice
        q[i] = ld_stream_v4(vec0 + (size_t)v * 16);
      } else if (v < v1 && e0 >= 0 && e0 + E <= V) {
        q[i] = ld_stream_v4(vec0 + (size_t)v * 16);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = BF16 ? 0xFF80FF80u : 0xFF800000u;
        if (v < v1) {
#pragma unroll
          for (int k = 0; k < E; ++k) {
            if (e0 + k < 0 || e0 + k >= V) continue;
            if (BF16) {
              const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(base) + e0 + k);
              w[k / 2] = (k & 1) ? (w[k / 2] & 0xFFFFu) | (h << 16) : (w[k / 2] & 0xFFFF0000u) | h;
            } else {
              w[k % 4] = __ldg(reinterpret_cast<const uint32_t*>(base) + e0 + k);
            }
          }
        }
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  uint4 cur[U], nxt[U];
  fetch(v0, cur);
  float tau = -INFINITY;  // nothing below it can be an alternative
  int listed = 0;         // keys in the warp's list
  lp_key_t tau_key = 0;   // the warp's own k-th best: keys must be above it
  const int keep = 2 * top + 4 < kLpKeep ? 2 * top + 4 : kLpKeep;  // a late cut leaves the threshold low
  // the elements of a round at or above tau, to the warp's list
  auto filter = [&](int r, const float (&x)[kLpElems]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = r + i * kLpThreads + tid;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const int e = v * E - lead + k;
        const lp_key_t key = lp_key(x[i * E + k], e);
        const bool in = x[i * E + k] >= tau && key > tau_key && v < v1 && e >= 0 && e < V;
        const uint32_t votes = __ballot_sync(0xffffffffu, in);
        if (in) s.list[warp][listed + __popc(votes & ((1u << lane) - 1))] = key;
        listed += __popc(votes);
      }
    }
    __syncwarp();
    if (listed > keep) {
      listed = lp_cut(s.list[warp], s.cut[warp], listed, top);
      if (listed == top) {
        tau_key = s.list[warp][top - 1];
        if (lane == 0) atomicMax(&s.tau, (uint32_t)(tau_key >> 32));
      }
    }
  };
  auto use = [&](int r, const uint4 (&q)[U], bool first) {
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
      const lp2 f2(f, f);
      run_u = mul2(f2, fma2(lp2(d, d), run_z, run_u));
      run_z = mul2(f2, run_z);
      run_m = bm;
    }
    const float m = run_m == -INFINITY ? 0.0f : run_m;
    const lp2 m2(-m, -m), l2(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < kLpElems; k += 2) {
      const lp2 d2 = add2(lp2(x[k], x[k + 1]), m2);
      float d0, d1, s0, s1;
      mul2(d2, l2).get(s0, s1);
      d2.get(d0, d1);
      const lp2 e2(lp_ex2(s0), lp_ex2(s1));
      run_z = add2(run_z, e2);                                                // a NaN or +infinity stays in z
      run_u = fma2(e2, lp2(fmaxf(d0, -1000.0f), fmaxf(d1, -1000.0f)), run_u);  // 0 x -infinity of a masked logit is 0
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
    if (top > 0) {
      if (first) {
        tau = lp_kth(bm, top);
        if (lane == 0 && tau > -INFINITY) atomicMax(&s.tau, lp_order(tau));
      } else {
        const uint32_t o = *reinterpret_cast<volatile uint32_t*>(&s.tau);
        if (o) tau = fmaxf(tau, lp_key_value((lp_key_t)o << 32));
      }
      if (__any_sync(0xffffffffu, bm >= tau)) filter(r, x);
    }
  };

  for (int r = v0; r < v1; r += kStep) {
    if (r + kStep < v1) fetch(r + kStep, nxt);
    use(r, cur, r == v0);
#pragma unroll
    for (int i = 0; i < U; ++i) cur[i] = nxt[i];
  }
  if (top > 0) {  // the warps' best, joined by the first warp
    const int n = lp_cut(s.list[warp], s.cut[warp], listed, top);
    if (lane < top) s.best[warp * top + lane] = lane < n ? s.list[warp][lane] : 0;
    if (tid < top) s.cut[0][tid] = 0;  // (lp_cut is done with it) a slice may hold fewer than k
    __syncthreads();
    lp_merge(s.best, s.cut[0], kLpWarps * top, top);
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
    const lp_key_t key = s.cut[0][tid];
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
    if (ctas > 1) lp_merge(s.inbox, s.cut[0], (int)ctas * top, top);
    if (tid < top) {
      const lp_key_t key = s.cut[0][tid];
      p.top_id[row * top + tid] = bad ? -1 : (int)~(uint32_t)key;
      p.top_val[row * top + tid] = bad ? nanv : logp(lp_key_value(key));
    }
  }
}

// CTAs per row: enough for four on every SM, of at least one round each.
static int lp_cluster(int N, int V) {
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  const int rounds = (V + kLpThreads * kLpElems - 1) / (kLpThreads * kLpElems);
  int c = 1;
  while (c < kLpMaxCluster && 2 * c <= rounds && (int64_t)N * c < (int64_t)4 * sms) c *= 2;
  return c;
}

template <bool BF16>
static cudaError_t launch_logprobs(const LogprobParams& p, int N, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(LpShared));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(logprobs_kernel<BF16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    allowed[dev] = 1;
  }
  const int ctas = lp_cluster(N, p.V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)N * ctas));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = sizeof(LpShared);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16>, p);
}

}  // namespace ft

extern "C" {

int ft_logprobs(const void* logits, int dtype, int64_t row_stride, int N, int V, const int32_t* targets, int top_k,
                float* logprob, float* entropy, int32_t* rank, int32_t* top_ids, float* top_logprobs,
                int32_t* dev_status, ft_stream stream) {
  if (dtype != FT_BF16 && dtype != FT_F32) return FT_ERR_INVALID_ARG;
  if (N < 0 || V < 1 || top_k < 0 || row_stride < V) return FT_ERR_INVALID_ARG;
  if (top_k > ft::kLpMaxTop || top_k > V) return FT_ERR_UNSUPPORTED;
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
