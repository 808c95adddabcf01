// Causal attention of packed prompts over their own BF16 rows.
#include <algorithm>

#include "ft_internal.cuh"

namespace ft {

struct PromptParams {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const int32_t* cu;
  int32_t* status;
  int B, total, max_len, nkv, G;
  float scale;  // x log2(e)
};

// A warp per row and query head, one key at a time.
template <int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptParams p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, nq = p.nkv * p.G;
  const int64_t warp = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t t = warp / nq;
  const int h = (int)(warp % nq);
  if (t >= p.total) return;
  int first = -1;
  for (int b = 0; b < p.B; ++b) {
    const int a = p.cu[b], z = p.cu[b + 1];
    if (a < 0 || z < a || z > p.total || z - a > p.max_len) {
      set_status(p.status, FT_DEV_RANGE);
    } else if (t >= a && t < z) {
      first = a;
    }
  }
  if (first < 0) return;
  float q[N], o[N] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = bf16_bits_to_f32(p.q[t * p.q_stride + h * D + lane + 32 * i]) * p.scale;
  for (int64_t j = first; j <= t; ++j) {
    float s = 0.0f, v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s = fmaf(q[i], bf16_bits_to_f32(p.k[j * p.k_stride + h / p.G * D + lane + 32 * i]), s);
      v[i] = bf16_bits_to_f32(p.v[j * p.v_stride + h / p.G * D + lane + 32 * i]);
    }
    s = warp_sum(s);
    const float to = fmaxf(m, s), f = to == m ? 1.0f : exp2f(m - to), e = exp2f(s - to);
    m = to;
    l = fmaf(l, f, e);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], f, e * v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) p.o[t * p.o_stride + h * D + lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] / l));
}

constexpr int kPromptMaxB = 8192;

}  // namespace ft

extern "C" {

int ft_attn_prompt_bf16(const ft_block_cfg* c, const uint16_t* q_bf16, int64_t q_stride, const uint16_t* k_bf16,
                        int64_t k_stride, const uint16_t* v_bf16, int64_t v_stride, const int32_t* cu_seqlens, int B,
                        int total, int max_len, float scale, uint16_t* o_bf16, int64_t o_stride, int32_t* dev_status,
                        ft_stream stream) {
  const int st = ft_host::check_cfg(c);
  if (st != FT_OK) return st;
  if (B < 1 || total < 0 || max_len < 1 || !(scale > 0.0f) || !(scale < 3e38f)) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  const int64_t row_q = (int64_t)c->n_q * c->head_dim, row_k = (int64_t)c->n_kv * c->head_dim;
  if (!q_bf16 || !k_bf16 || !v_bf16 || !cu_seqlens || !o_bf16 || q_stride < row_q || o_stride < row_q || k_stride < row_k ||
      v_stride < row_k)
    return FT_ERR_INVALID_ARG;
  if (!ft_host::aligned16(k_bf16) || !ft_host::aligned16(v_bf16) || k_stride % 8 || v_stride % 8) return FT_ERR_INVALID_ARG;
  if (B > ft::kPromptMaxB || (int64_t)total * (c->n_q / c->n_kv) > INT32_MAX) return FT_ERR_UNSUPPORTED;
  ft::PromptParams p = {};
  p.q = q_bf16, p.k = k_bf16, p.v = v_bf16, p.o = o_bf16;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride, p.o_stride = o_stride;
  p.cu = cu_seqlens;
  p.status = dev_status;
  p.B = B;
  p.total = total;
  p.max_len = max_len;
  p.nkv = c->n_kv;
  p.G = c->n_q / c->n_kv;
  p.scale = scale * 1.44269504088896341f;
  const int64_t blocks = ((int64_t)total * c->n_q + 3) / 4;
  if (blocks > INT32_MAX) return FT_ERR_UNSUPPORTED;
  if (c->head_dim == 128) ft::prompt_rows_kernel<128><<<(unsigned)blocks, 128, 0, (cudaStream_t)stream>>>(p);
  else ft::prompt_rows_kernel<64><<<(unsigned)blocks, 128, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
