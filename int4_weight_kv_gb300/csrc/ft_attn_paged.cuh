// What the kernels of attention over the paged 4-bit cache share.
//
//   o = H sum_j softmax_j(scale (H q) . K^_j) V^_j   over positions j <= the token's
//
// with K^_j = ks_j x codes and V^_j = vs_j x codes.  In log2 units, with lv_j =
// log2(vs_j) and t_j = scale log2(e) (H q) . K^_j + lv_j:
//   p_j = 2^(t_j - m),   o = (sum_j p_j codes_j) / (sum_j p_j / vs_j),
// so the V scales never multiply the matrix product's operand P: it stays within
// FP16 whatever the scales are, and one FMA applies both scales to a score.
#pragma once

#include "ft_paged.cuh"

namespace ft {

constexpr float kQUp = 64.0f;                 // query operand: q scale log2(e) x 64 (keeps q / 16 out of FP16's subnormals)
constexpr float kKsUp = 262144.0f;            // 2^24 (codes are x 2^-24) / 64
constexpr float kOUp = 16777216.0f;           // 2^24
constexpr float kPBias = 10.0f;               // P = 2^(t - m + 10): FP16 normals down to 2^-24 of the largest weight
constexpr float kPLazy = 4.0f;                // the running max moves when a score passes it by 2^4 (P < 2^14 + rounding)
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100: smaller V scales count as this (their values are ~0)
// Scales from here on (2^110, as BF16 bits) make a row that sees them NaN, as those that are not finite
// do: past them the factors of scores and sums of weights leave FP32.
constexpr uint32_t kTooLarge = 0x7680u;
// An entry whose V is zero (scale 0) weighs in the sum of weights alone, with lv = -60.  A weight is lost
// where 2^(t - m) passes below FP32's 2^-126: V scales 2^100 apart leave 2^26 for the softmax's own ratio,
// more than FP32's digits, and 2^40 is as far above an entry without values.  Values of 2^-70 beside one
// still have P = 1 at equal scores, 2^14 above FP16's subnormals.
constexpr uint32_t kNoScaleExp = 67u;           // exponent of 2^-60
constexpr float kNoScale = 8.6736173798840355e-19f;  // 2^-60

struct AttnPagedParams {
  const uint8_t* pages;
  PagedLayout L;
  const uint16_t* q;
  uint16_t* o;
  int64_t q_stride, o_stride;
  const int32_t *cu, *kv_len, *table;
  int32_t* status;
  int table_stride, B, total_q, max_q, G, hb;
  float qscale, norm;  // scale log2(e) kQUp; 1 / sqrt(hb)
};

// One request's length, checked: 0 (every row empty: zeros) where it is negative, passes the table
// row or is within a tile of 2^31.
__device__ __forceinline__ int attn_length(const AttnPagedParams& p, int b, int32_t* status) {
  const int kv = p.kv_len[b];
  if (kv >= 0 && kv <= INT32_MAX - 256 && ((kv + p.L.psize - 1) >> p.L.pshift) <= p.table_stride) return kv;
  set_status(status, FT_DEV_CAPACITY);
  return 0;
}

// One request's rows and length, checked (conditions to status, which may be NULL); false:
// nothing of it is computed.
__device__ __forceinline__ bool attn_request(const AttnPagedParams& p, int b, int32_t* status, int& row0, int& n, int& kv) {
  row0 = p.cu[b];
  n = p.cu[b + 1] - row0;
  kv = attn_length(p, b, status);
  if (row0 < 0 || n < 0 || row0 > p.total_q - n || n > p.max_q) {
    set_status(status, FT_DEV_RANGE);
    return false;
  }
  return true;
}

// MUFU operations without the denormal handling of the library functions.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Joins n partials (max, sum, 2 unused, accumulator) of one row and stores it, a warp (or a CTA of
// W warps) per row, eight partials' loads in flight in each; row(i) is partial i, `up` the
// accumulators' factor.
template <int D, int W = 1, typename Row>
__device__ __forceinline__ void join_row(const AttnPagedParams& p, int n, Row row, float up, uint16_t* dst) {
  constexpr int CH = D / 32, kBatch = 8;  // channels CH lane .. + CH - 1 of each lane
  const int lane = threadIdx.x & 31, warp = W > 1 ? threadIdx.x >> 5 : 0;
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(row(i)));
  M = warp_max(M);
  float lt = 0.0f, o[CH] = {};
  for (int c = kBatch * warp; c < n; c += kBatch * W) {
    float2 ml[kBatch];
    float x[kBatch][CH];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (c + i >= n) continue;
      const float* q = row(c + i);
      ml[i] = __ldcg(reinterpret_cast<const float2*>(q));
      if constexpr (D == 128) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(q + 4) + lane);
        x[i][0] = f.x, x[i][1] = f.y, x[i][2] = f.z, x[i][3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(q + 4) + lane);
        x[i][0] = f.x, x[i][1] = f.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (c + i >= n) continue;
      const float f = ml[i].x == M ? 1.0f : ex2(ml[i].x - M);
      lt = fmaf(f, ml[i].y, lt);
#pragma unroll
      for (int k = 0; k < CH; ++k) o[k] = fmaf(f, x[i][k], o[k]);
    }
  }
  if constexpr (W > 1) {  // the warps' sums, in their order
    __shared__ float sums[W][D + 1];
#pragma unroll
    for (int k = 0; k < CH; ++k) sums[warp][CH * lane + k] = o[k];
    if (lane == 0) sums[warp][D] = lt;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      lt += sums[w][D];
#pragma unroll
      for (int k = 0; k < CH; ++k) o[k] += sums[w][CH * lane + k];
    }
  }
  const float inv = lt == 0.0f ? 0.0f : up / lt;  // a row that sees nothing: zeros
  // the rotation of neighbouring channels, strides 1 (and 2) in the lane, the others across lanes
#pragma unroll
  for (int k = 0; k < CH; ++k) o[k] *= inv;
#pragma unroll
  for (int s = 1; s < CH; s <<= 1) {
    if (s >= p.hb) break;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if (k & s) continue;
      const float a = o[k], c = o[k + s];
      o[k] = a + c;
      o[k + s] = a - c;
    }
  }
  for (int s = 1; CH * s < p.hb; s <<= 1) {
    const float sign = (lane & s) ? -1.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) o[k] = fmaf(sign, o[k], __shfl_xor_sync(0xffffffffu, o[k], s));
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) dst[CH * lane + k] = __bfloat16_as_ushort(__float2bfloat16_rn(o[k] * p.norm));
}

// Requests with many rows (ft_attn_tiles.cu); a workspace of attn_tiles_ws bytes.
size_t attn_tiles_ws(int nkv, int G, int head_dim, int B, int total_q);
int64_t attn_tiles_ctas(const AttnPagedParams& p);
cudaError_t launch_attn_tiles(const AttnPagedParams& p, int head_dim, void* workspace, cudaStream_t st);

}  // namespace ft
