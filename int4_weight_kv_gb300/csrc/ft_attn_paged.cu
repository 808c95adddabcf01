// Attention of any number of new tokens per request over the paged 4-bit cache.
//
//   o = H sum_j softmax_j(scale (H q) . K^_j) V^_j   over positions j <= the token's
//
// with K^_j = ks_j x codes and V^_j = vs_j x codes.  In log2 units, with lv_j =
// log2(vs_j) and t_j = scale log2(e) (H q) . K^_j + lv_j:
//   p_j = 2^(t_j - m),   o = (sum_j p_j codes_j) / (sum_j p_j / vs_j),
// so the V scales never multiply the matrix product's operand P: it stays within
// FP16 whatever the scales are, and one FMA applies both scales to a score.
#include <algorithm>

#include "ft_paged.cuh"

namespace ft {

constexpr float kQUp = 64.0f;                 // query operand: q scale log2(e) x 64 (keeps q / 16 out of FP16's subnormals)
constexpr float kKsUp = 262144.0f;            // 2^24 (codes are x 2^-24) / 64
constexpr float kOUp = 16777216.0f;           // 2^24
constexpr float kPBias = 10.0f;               // P = 2^(t - m + 10): FP16 normals down to 2^-24 of the largest weight
constexpr float kPLazy = 4.0f;                // the running max moves when a score passes it by 2^4 (P < 2^14 + rounding)
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100: smaller V scales count as this (their values are ~0)

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

// One request's rows and length, checked; false: nothing of it is computed.
__device__ __forceinline__ bool attn_request(const AttnPagedParams& p, int b, int& row0, int& n, int& kv) {
  row0 = p.cu[b];
  n = p.cu[b + 1] - row0;
  kv = p.kv_len[b];
  if (row0 < 0 || n < 0 || row0 > p.total_q - n || n > p.max_q) {
    set_status(p.status, FT_DEV_RANGE);
    return false;
  }
  if (kv < 0 || ((kv + (int64_t)p.L.psize - 1) >> p.L.pshift) > p.table_stride) {
    set_status(p.status, FT_DEV_CAPACITY);
    kv = 0;  // every row empty: zeros
  }
  return true;
}

constexpr int kApWarps = 4;

// Eight rows (token, head of the group) of one request and KV head per CTA; warps
// take 16-position tiles in turn.  S = K q (rows positions, columns the 8 rows),
// O^T = V^T P.
template <int D>
__global__ void __launch_bounds__(kApWarps * 32) attn_paged_kernel(const AttnPagedParams p) {
  constexpr int KT = D / 16, NPL = D / 32, NJ = D / 32, PW = D + 4;
  __shared__ float qt[8][D];
  __shared__ float part[kApWarps][8][PW];  // max, sum, acc
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, r0 = 8 * blockIdx.x;
  int row0, n, kv;
  if (!attn_request(p, b, row0, n, kv)) return;
  const int nrow = n * p.G - r0;
  if (nrow <= 0) return;
  for (int r = warp; r < 8; r += kApWarps) {
    float v[NPL];
    const int tok = (r0 + r) / p.G, hh = (r0 + r) - tok * p.G;
    const uint16_t* src = p.q + (row0 + tok) * p.q_stride + (int64_t)(h * p.G + hh) * D;
    bool bad = false;
#pragma unroll
    for (int m = 0; m < NPL; ++m) v[m] = r < nrow ? bf16_bits_to_f32(src[lane + 32 * m]) : 0.0f;
    warp_fwht<NPL>(v, p.hb);
#pragma unroll
    for (int m = 0; m < NPL; ++m) {
      const int c = lane + 32 * m;
      const float x = v[m] * p.qscale;
      bad |= !(fabsf(x) <= 65504.0f);
      qt[r][c] = (c & 8) ? x * 0.0625f : x;
    }
    if (bad) set_status(p.status, FT_DEV_RANGE);
  }
  __syncthreads();
  uint32_t bq[KT][2];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int c = 16 * kt + 2 * tig;
    const __half2 lo = __floats2half2_rn(qt[g][c], qt[g][c + 1]), hi = __floats2half2_rn(qt[g][c + 8], qt[g][c + 9]);
    bq[kt][0] = *reinterpret_cast<const uint32_t*>(&lo);
    bq[kt][1] = *reinterpret_cast<const uint32_t*>(&hi);
  }
  // last visible position of this lane's two rows; -1: none
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 2 * tig + i;
    lim[i] = 2 * tig + i < nrow ? kv - n + r / p.G : -1;
  }
  const int last = kv - n + (r0 + min(nrow, 8) - 1) / p.G;  // of any row

  float acc[KT][4];
#pragma unroll
  for (int mt = 0; mt < KT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.0f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  for (int tile = warp; 16 * tile <= last; tile += kApWarps) {
    const int p0 = 16 * tile, pin = p0 & (p.L.psize - 1);
    const int page = p.table[(size_t)b * p.table_stride + (p0 >> p.L.pshift)];
    if (page < 0 || page >= p.L.npages) {
      if (lane == 0) set_status(p.status, FT_DEV_RANGE);
      continue;
    }
    const uint8_t* blk = p.pages + paged_block(p.L, page, h);
    uint32_t kw[2][NJ], vw[2][NJ];
    const uint8_t* k0 = blk + (pin + g) * (D / 2) + tig * (D / 8);
    const uint8_t* v0 = blk + p.L.voff + (pin / 2 + tig) * D + (g ^ paged_v_turn<D>(tig)) * (D / 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (D == 128) {
        const uint4 a = ld_stream_v4(k0 + i * 8 * (D / 2)), c = ld_stream_v4(v0 + i * 4 * D);
        kw[i][0] = a.x, kw[i][1] = a.y, kw[i][2] = a.z, kw[i][3] = a.w;
        vw[i][0] = c.x, vw[i][1] = c.y, vw[i][2] = c.z, vw[i][3] = c.w;
      } else {
        const uint2 a = ld_stream_v2(k0 + i * 8 * (D / 2)), c = ld_stream_v2(v0 + i * 4 * D);
        kw[i][0] = a.x, kw[i][1] = a.y;
        vw[i][0] = c.x, vw[i][1] = c.y;
      }
    }
    const uint32_t sc0 = ld_stream_u32(blk + p.L.soff + 4 * (pin + g)), sc1 = ld_stream_u32(blk + p.L.soff + 4 * (pin + g + 8));
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t lo[4], hi[4];
      paged_word(kw[0][j], lo);
      paged_word(kw[1][j], hi);
      const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
      mma_f16(s, a0, bq[2 * j][0], bq[2 * j][1]);
      mma_f16(s, a1, bq[2 * j + 1][0], bq[2 * j + 1][1]);
    }
    const float ks0 = __uint_as_float(sc0 << 16) * kKsUp, ks1 = __uint_as_float(sc1 << 16) * kKsUp;
    const float vs0 = fmaxf(__uint_as_float(sc0 & 0xFFFF0000u), kMinScale);
    const float vs1 = fmaxf(__uint_as_float(sc1 & 0xFFFF0000u), kMinScale);
    const float lv0 = __log2f(vs0), lv1 = __log2f(vs1), rs0 = __frcp_rn(vs0), rs1 = __frcp_rn(vs1);
    const int pa = p0 + g, pb = pa + 8;
    const bool in[4] = {pa <= lim[0], pa <= lim[1], pb <= lim[0], pb <= lim[1]};
    float x[4] = {fmaf(s[0], ks0, lv0), fmaf(s[1], ks0, lv0), fmaf(s[2], ks1, lv1), fmaf(s[3], ks1, lv1)};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = in[i] ? x[i] : -INFINITY;  // whatever the masked entry holds
    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, mx0 > m0 + kPLazy || mx1 > m1 + kPLazy)) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      const float f0 = m0 == n0 ? 1.0f : exp2f(m0 - n0), f1 = m1 == n1 ? 1.0f : exp2f(m1 - n1);
      m0 = n0, m1 = n1;
      l0 *= f0, l1 *= f1;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) acc[mt][0] *= f0, acc[mt][1] *= f1, acc[mt][2] *= f0, acc[mt][3] *= f1;
    }
    const float u0 = m0 == -INFINITY ? 0.0f : m0 - kPBias, u1 = m1 == -INFINITY ? 0.0f : m1 - kPBias;
    const float e[4] = {exp2f(x[0] - u0), exp2f(x[1] - u1), exp2f(x[2] - u0), exp2f(x[3] - u1)};
    // a masked entry's scale may hold anything: it adds no weight
    l0 += (in[0] ? e[0] * rs0 : 0.0f) + (in[2] ? e[2] * rs1 : 0.0f);
    l1 += (in[1] ? e[1] * rs0 : 0.0f) + (in[3] ? e[3] * rs1 : 0.0f);
    const __half2 pa2 = __floats2half2_rn(e[0], e[1]), pb2 = __floats2half2_rn(e[2], e[3]);
    const uint32_t b0 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&pa2));
    const uint32_t b1 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&pb2));
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t lo[4], hi[4];
      paged_word(vw[0][j], lo);
      paged_word(vw[1][j], hi);
      const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]}, a1[4] = {lo[2], lo[3], hi[2], hi[3]};
      mma_f16(acc[2 * j], a0, b0, b1);
      mma_f16(acc[2 * j + 1], a1, b0, b1);
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, o);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  }
  float* w0 = part[warp][2 * tig];
  float* w1 = part[warp][2 * tig + 1];
  if (g == 0) w0[0] = m0, w0[1] = l0, w1[0] = m1, w1[1] = l1;
#pragma unroll
  for (int mt = 0; mt < KT; ++mt) {
    const int c = 16 * mt + g;
    w0[4 + c] = acc[mt][0], w1[4 + c] = acc[mt][1];
    w0[4 + c + 8] = acc[mt][2] * 0.0625f, w1[4 + c + 8] = acc[mt][3] * 0.0625f;
  }
  __syncthreads();
  for (int r = warp; r < min(8, nrow); r += kApWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kApWarps; ++w) M = fmaxf(M, part[w][r][0]);
    float l = 0.0f, o[NPL] = {};
#pragma unroll
    for (int w = 0; w < kApWarps; ++w) {
      const float m = part[w][r][0], f = m == M ? 1.0f : exp2f(m - M);
      l = fmaf(f, part[w][r][1], l);
#pragma unroll
      for (int m2 = 0; m2 < NPL; ++m2) o[m2] = fmaf(f, part[w][r][4 + lane + 32 * m2], o[m2]);
    }
    const float inv = l == 0.0f ? 0.0f : kOUp / l;  // a row that sees nothing: zeros
#pragma unroll
    for (int m2 = 0; m2 < NPL; ++m2) o[m2] *= inv;
    warp_fwht<NPL>(o, p.hb);
    const int tok = (r0 + r) / p.G, hh = (r0 + r) - tok * p.G;
    uint16_t* dst = p.o + (row0 + tok) * p.o_stride + (int64_t)(h * p.G + hh) * D;
#pragma unroll
    for (int m2 = 0; m2 < NPL; ++m2) dst[lane + 32 * m2] = __bfloat16_as_ushort(__float2bfloat16_rn(o[m2]));
  }
}

}  // namespace ft

extern "C" {

size_t ft_attn_paged_workspace_bytes(const ft_block_cfg* c, int B, int total_q, int max_q) {
  if (ft_host::check_cfg(c) != FT_OK || B < 1 || total_q < 0 || max_q < 1) return 0;
  return 16;
}

int ft_attn_paged_int4(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const uint16_t* q_bf16,
                       int64_t q_stride, const int32_t* cu_seqlens, const int32_t* kv_len, const int32_t* block_table,
                       int table_stride, int B, int total_q, int max_q, float scale, uint16_t* o_bf16, int64_t o_stride,
                       void* workspace, size_t ws_bytes, int32_t* dev_status, ft_stream stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (B < 1 || total_q < 0 || max_q < 1 || table_stride < 1 || !(scale > 0.0f) || !(scale < 3e38f))
    return FT_ERR_INVALID_ARG;
  if (total_q == 0) return FT_OK;
  const int64_t row = (int64_t)c->n_q * c->head_dim;
  if (!q_bf16 || !o_bf16 || !cu_seqlens || !kv_len || !block_table || !workspace || q_stride < row || o_stride < row)
    return FT_ERR_INVALID_ARG;
  if (!ft_host::aligned16(workspace)) return FT_ERR_INVALID_ARG;
  if (ws_bytes < ft_attn_paged_workspace_bytes(c, B, total_q, max_q)) return FT_ERR_WORKSPACE;
  if (B > 65535) return FT_ERR_UNSUPPORTED;
  ft::AttnPagedParams p = {};
  p.pages = static_cast<const uint8_t*>(pages);
  p.L = ft::paged_layout(*c, n_pages, page_size);
  p.q = q_bf16;
  p.o = o_bf16;
  p.q_stride = q_stride;
  p.o_stride = o_stride;
  p.cu = cu_seqlens;
  p.kv_len = kv_len;
  p.table = block_table;
  p.status = dev_status;
  p.table_stride = table_stride;
  p.B = B;
  p.total_q = total_q;
  p.max_q = std::min(max_q, total_q);
  p.G = c->n_q / c->n_kv;
  p.hb = c->had_block;
  p.qscale = scale * 1.44269504088896341f * ft::kQUp;
  p.norm = ft::paged_norm(c->had_block);
  const int64_t rb = ((int64_t)p.max_q * p.G + 7) / 8;
  const dim3 grid((unsigned)rb, c->n_kv, B);
  if (c->head_dim == 128)
    ft::attn_paged_kernel<128><<<grid, ft::kApWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else
    ft::attn_paged_kernel<64><<<grid, ft::kApWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
