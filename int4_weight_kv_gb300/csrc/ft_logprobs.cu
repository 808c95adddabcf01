// Log probabilities of given tokens, with the distribution's entropy, the token's
// rank and the k most probable alternatives.
//
//   m = max x, z = sum 2^((x - m) log2 e):  log z + m is the normaliser,
//   entropy = log z - sum e (x - m) / z.
//
// One CTA per row.  Alternatives are ordered by a 64-bit key (the value as an ordered
// integer, then the lower index), so ties have one answer whatever order the row is
// read in.
#include <algorithm>

#include "ft_internal.cuh"

namespace ft {

constexpr int kLpThreads = 512, kLpMaxTop = 32;

struct LogprobParams {
  const void* x;
  int64_t stride;
  const int32_t* target;
  float *logprob, *entropy, *top_val;
  int32_t *rank, *top_id, *status;
  int V, top;
};

template <bool BF16>
__device__ __forceinline__ float lp_load(const void* x, int64_t i) {
  if (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(x)[i]);
  return static_cast<const float*>(x)[i];
}
// Larger key: larger value (-0 = +0), then lower index.
__device__ __forceinline__ unsigned long long lp_key(float v, int i) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float lp_key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

template <typename T, typename F>
__device__ __forceinline__ T lp_block_reduce(T v, F op, T* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  v = sh[0];
  for (int w = 1; w < kLpThreads / 32; ++w) v = op(v, sh[w]);
  __syncthreads();
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobParams p) {
  __shared__ float shf[kLpThreads / 32];
  __shared__ unsigned long long shk[kLpThreads / 32];
  const int tid = threadIdx.x, V = p.V;
  const int64_t row = blockIdx.x, at = row * p.stride;
  const int t = p.target ? p.target[row] : -1;
  const bool has = t >= 0 && t < V;
  const float xt = has ? lp_load<BF16>(p.x, at + t) : 0.0f;
  const auto fadd = [](float a, float b) { return a + b; };
  float m = -INFINITY, nan = 0.0f;
  for (int i = tid; i < V; i += kLpThreads) {
    const float v = lp_load<BF16>(p.x, at + i);
    m = fmaxf(m, v);
    if (!(v < INFINITY)) nan = 1.0f;
  }
  m = lp_block_reduce(m, [](float a, float b) { return fmaxf(a, b); }, shf);
  nan = lp_block_reduce(nan, fadd, shf);
  const bool bad = nan > 0.0f || m == -INFINITY;  // a NaN or +infinity, or nothing that is possible
  float z = 0.0f, u = 0.0f, above = 0.0f;
  for (int i = tid; i < V && !bad; i += kLpThreads) {
    const float v = lp_load<BF16>(p.x, at + i), d = fmaxf(v - m, -1e4f), e = expf(d);
    z += e;
    u = fmaf(e, d, u);
    above += (v > xt || (v == xt && i < t)) ? 1.0f : 0.0f;
  }
  z = lp_block_reduce(z, fadd, shf);
  u = lp_block_reduce(u, fadd, shf);
  above = lp_block_reduce(above, fadd, shf);
  const float lz = logf(z), lse = m + lz, nanv = __int_as_float(0x7FC00000);
  if (tid == 0) {
    if (bad || (t != -1 && !has)) set_status(p.status, FT_DEV_RANGE);
    if (p.logprob) p.logprob[row] = t == -1 ? 0.0f : (bad || !has) ? nanv : xt - lse;
    if (p.entropy) p.entropy[row] = bad ? nanv : lz - u / z;
    if (p.rank) p.rank[row] = (bad || !has) ? -1 : (int)above;
  }
  unsigned long long prev = ~0ull;
  for (int k = 0; k < p.top; ++k) {
    unsigned long long best = 0ull;
    for (int i = tid; i < V && !bad; i += kLpThreads) {
      const unsigned long long key = lp_key(lp_load<BF16>(p.x, at + i), i);
      if (key < prev && key > best) best = key;
    }
    best = lp_block_reduce(best, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; }, shk);
    if (tid == 0) {
      p.top_id[row * p.top + k] = bad ? -1 : (int)~(uint32_t)best;
      p.top_val[row * p.top + k] = bad ? nanv : lp_key_value(best) - lse;
    }
    prev = best;
  }
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
  if (dtype == FT_BF16)
    ft::logprobs_kernel<true><<<N, ft::kLpThreads, 0, (cudaStream_t)stream>>>(p);
  else
    ft::logprobs_kernel<false><<<N, ft::kLpThreads, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
