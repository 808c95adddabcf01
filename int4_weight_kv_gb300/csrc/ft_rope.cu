// Rows of the fused projection made ready for the cache and for attention: per-head RMS norms and the
// position rotation of q and k, and the placement of k and v in the paged 4-bit cache on the way.
//
//   y = gamma x / sqrt(mean x^2 + eps),   z_i = y_i cos a - y_(i+d/2) sin a,  z_(i+d/2) = y_(i+d/2) cos a + y_i sin a
//
// Every byte is moved once.  Measured, 32 heads over 8 of 128: norm and rotation of 17k tokens 62 us, 83% of the copy rate
// (bound by HBM), of 32 tokens 3.1; placement of 9k tokens' k and v, with q's on the way and norms, 56 us, 1.9 times what
// the bytes take: neither the issue slots (50%) nor HBM (39%) are at their end, there is too little in flight (27% of the
// warps resident, for their 80 registers, of which 88 bytes are spilled; 2.5 waves of CTAs).
#include <algorithm>

#include "ft_paged.cuh"

namespace ft {

// D / 16 lanes per row: lane c owns channels 8 c .. 8 c + 7 and d/2 + 8 c .. d/2 + 8 c + 7, two 16-byte
// pieces, so that the pairs of the rotation meet in one lane.  A CTA has 4 (8) consecutive tokens, their angles in
// shared memory, and a warp of its four goes through `per` heads of them.
// Heads at most, 4 / 8 / 12 / 16 (us): rows of 17k tokens 67.6 / 63.2 / 61.3 / 61.3, placement of 9k with reading back
// 73.1 / 71.5 / 69.9 / 69.9.
constexpr int kRopeThreads = 128, kRopeHeads = 12;
// tensors whose rows are at 16-byte boundaries
enum { kWideQ = 1, kWideK = 2, kWideV = 4, kWideQOut = 8, kWideKOut = 16 };

struct RopeRows {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const float *gamma_q, *gamma_k;
  const int32_t *pos, *slots;
  uint8_t* pages;
  PagedLayout L;
  int total, nq, nkv, heads, per, hb, wide;  // heads: nq q heads, then k, then (paged) v; per: those of a warp
  float norm, eps;
  int32_t* status;
  uint64_t turn[64];
};

// A lane's two pieces of a row, as they are.  Rows at 16-byte boundaries are told apart by the host.
template <int D>
__device__ __forceinline__ void rope_load(const uint16_t* src, bool wide, uint4 (&raw)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t* at = src + i * (D / 2);
    if (wide) {
      raw[i] = *reinterpret_cast<const uint4*>(at);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = (uint32_t)at[2 * k] | ((uint32_t)at[2 * k + 1] << 16);
      raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
__device__ __forceinline__ void rope_values(const uint4 (&raw)[2], f32x2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[4 * i + k] = f32x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  }
}
template <int D>
__device__ __forceinline__ void rope_store(uint16_t* dst, bool wide, const f32x2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t* at = dst + i * (D / 2);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      x[4 * i + k].get(a, b);
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if (wide) {
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) at[2 * k] = (uint16_t)w[k], at[2 * k + 1] = (uint16_t)(w[k] >> 16);
    }
  }
}

// H times the row, strides 1, 2, 4, ... in this order (as paged_fwht: the same rows give the same bits).
template <int D>
__device__ __forceinline__ void rope_fwht(f32x2 (&x)[8], int hb) {
  const f32x2 minus(-1.0f, -1.0f);
  if (hb > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      x[i].get(a, b);
      x[i] = f32x2(a + b, a - b);
    }
  }
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    if (2 * s >= hb) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & s) continue;
      const f32x2 a = x[i], b = x[i + s];
      x[i] = add2(a, b);
      x[i + s] = fma2(b, minus, a);
    }
  }
#pragma unroll
  for (int s = 1; s < D / 16; s <<= 1) {
    if (8 * s >= hb) break;
    const float sign = (threadIdx.x & s) ? -1.0f : 1.0f;
    const f32x2 sign2(sign, sign);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      x[i].get(a, b);
      const f32x2 o(__shfl_xor_sync(0xffffffffu, a, s), __shfl_xor_sync(0xffffffffu, b, s));
      x[i] = fma2(sign2, x[i], o);
    }
  }
  if (hb == D) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = x[i], b = x[i + 4];
      x[i] = add2(a, b);
      x[i + 4] = fma2(b, minus, a);
    }
  }
}

// One row rotated by H, quantised and stored at its slot (-1: not stored).
template <int D>
__device__ __forceinline__ void rope_place(const RopeRows& p, f32x2 (&x)[8], bool is_v, int h, int slot) {
  constexpr int LV = D / 16, NJ = D / 32;
  const int c = threadIdx.x % LV, e = c % 4, j = c / 4;
  rope_fwht<D>(x, p.hb);
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    x[i].get(a, b);
    am = max_nan(am, max_nan(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = 1; o < LV; o <<= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (!(am < INFINITY) && slot >= 0) set_status(p.status, FT_DEV_RANGE);
  const uint16_t sb = quant_scale_bits(am * p.norm);
  const float s = bf16_bits_to_f32(sb);
  // codes by a reciprocal, those near a boundary decided exactly (as append_paged_kernel)
  const float r = s >= 1e-30f ? p.norm * __frcp_rn(s) : 0.0f;
  const f32x2 r2(r, r), magic2(kMagic, kMagic), minus(-1.0f, -1.0f);
  const float far = r > 0.0f || s == 0.0f ? 0.5f - 7.0f * 4.76837158203125e-07f : -1.0f;  // 7 x 2^-21
  const int mag_at = (e & 1) * 3 + (e >> 1) * 8, neg_at = 8 * (e >> 1) + (e & 1);  // the latter: places below bit 15
  uint32_t w[8];  // this lane's value of words 2 i, 2 i + 1 of group j (i < 4), and of group j + NJ / 2
  f32x2 u[8];
  float near = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b, d0, d1;
    x[i].get(a, b);
    const f32x2 mag(fabsf(a), fabsf(b));
    u[i] = fma2(mag, r2, magic2);
    fma2(mag, r2, fma2(u[i], minus, magic2)).get(d0, d1);
    near = fmaxf(near, fmaxf(fabsf(d0), fabsf(d1)));
  }
  if (near >= far) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[2], m[2];
      x[i].get(v[0], v[1]);
      u[i].get(m[0], m[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float a = fabsf(v[k]), code = m[k] - kMagic;
        if (fabsf(fmaf(a, r, -code)) >= far) m[k] = kMagic + paged_edge(a * p.norm, s, code);
      }
      u[i] = f32x2(m[0], m[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b, m0, m1;
    x[i].get(a, b);
    u[i].get(m0, m1);
    w[i] = ((prmt(__float_as_uint(m0), __float_as_uint(m1), 0x5410u) & 0x00070007u) << mag_at) |
           ((prmt(__float_as_uint(a), __float_as_uint(b), 0x7632u) & 0x80008000u) >> neg_at);
  }
  // the four lanes of a group put their values together, lane e keeping words 2 e and 2 e + 1
  uint32_t k4[4], k2[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 4 * (i >> 1) + (i & 1);
    const uint32_t send = (e & 2) ? w[at] : w[at + 2], keep = (e & 2) ? w[at + 2] : w[at];
    k4[i] = keep | __shfl_xor_sync(0xffffffffu, send, 2);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t send = (e & 1) ? k4[2 * i] : k4[2 * i + 1], keep = (e & 1) ? k4[2 * i + 1] : k4[2 * i];
    k2[i] = keep | __shfl_xor_sync(0xffffffffu, send, 1);
  }
  const int pos = max(slot, 0) & (p.L.psize - 1);
  uint8_t* blk = p.pages + paged_block(p.L, max(slot, 0) >> p.L.pshift, h);
  if (!is_v) {
    if (slot >= 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<uint32_t*>(blk + paged_k_word<D>(pos, 2 * e, j + i * (NJ / 2))) = k2[i];
    }
  } else {
    // a pair's two positions in neighbouring groups of lanes: each side stores whole words
    const int other = __shfl_xor_sync(0xffffffffu, slot, LV);
    const bool odd = (slot & 1) != 0;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, prmt(k2[0], k2[1], odd ? 0x5410u : 0x7632u), LV);
    uint8_t* dst = blk + p.L.voff;
    if (slot >= 0 && other == (slot ^ 1)) {
      const uint32_t w0 = odd ? prmt(got, k2[0], 0x7610u) : prmt(k2[0], got, 0x5410u);
      const uint32_t w1 = odd ? prmt(got, k2[1], 0x7632u) : prmt(k2[1], got, 0x7610u);
      *reinterpret_cast<uint32_t*>(dst + paged_v_word<D>(pos & ~1, 2 * e + (odd ? 1 : 0), j)) = w0;
      *reinterpret_cast<uint32_t*>(dst + paged_v_word<D>(pos & ~1, 2 * e + (odd ? 1 : 0), j + NJ / 2)) = w1;
    } else if (slot >= 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint16_t*>(dst + paged_v_word<D>(pos, 2 * e, j + i * (NJ / 2))) = (uint16_t)k2[i];
        *reinterpret_cast<uint16_t*>(dst + paged_v_word<D>(pos, 2 * e + 1, j + i * (NJ / 2))) = (uint16_t)(k2[i] >> 16);
      }
    }
  }
  if (slot >= 0 && c == 0) *reinterpret_cast<uint16_t*>(blk + p.L.soff + 4 * pos + (is_v ? 2 : 0)) = sb;
}

// CTAs an SM, rows 6 / 7 / 8: 63.9 / 61.3 / 65.7 us for 17k tokens; placement 5 / 6 / 7: 75.5 / 69.9 / 75.0 for 9k.
template <int D, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads, PAGED ? 6 : 7) rope_rows_kernel(const __grid_constant__ RopeRows p) {
  constexpr int LV = D / 16, R = 32 / LV, W = kRopeThreads / 32;
  __shared__ __align__(16) float2 angles[R][D / 2 + 2];  // (cos, sin) of the CTA's tokens, each warp's share of them made by it
  griddep_serve();
  const int lane = threadIdx.x & 31, c = lane % LV, warp = threadIdx.x >> 5;
  const int chunks = (p.heads + W * p.per - 1) / (W * p.per), chunk = blockIdx.x % chunks;
  const int64_t t = (int64_t)(blockIdx.x / chunks) * R + lane / LV;
  const bool there = t < p.total;
  const int h0 = min((chunk * W + warp) * p.per, p.heads), h1 = min(h0 + p.per, p.heads), turned = p.nq + p.nkv;
  const int64_t row = there ? t : 0;  // (rows behind the last one read the first: nothing of them is stored)
  // the first head of each kind that this warp has, and the next one's bytes on their way
  auto source = [&](int hh) {
    return (hh < p.nq ? p.q + row * p.q_stride + hh * D
            : hh < turned ? p.k + row * p.k_stride + (hh - p.nq) * D
                          : p.v + row * p.v_stride + (hh - turned) * D) + 8 * c;
  };
  auto wide_of = [&](int hh) { return (p.wide & (hh < p.nq ? kWideQ : hh < turned ? kWideK : kWideV)) != 0; };
  uint4 raw[2];
  const uint16_t* src = source(h0 < p.heads ? h0 : 0);
  rope_load<D>(src, wide_of(h0 < p.heads ? h0 : 0), raw);
  if (chunk * W * p.per < turned) {
    const int pos = p.pos[row];
    float2* to = &angles[lane / LV][8 * c + 8 / W * warp];
#pragma unroll
    for (int k = 0; k < 8 / W; ++k) {
      const uint64_t a = (uint64_t)(int64_t)pos * p.turn[8 * c + 8 / W * warp + k];  // turns, modulo one
      float sn, cs;
      sincospif((float)(int32_t)(uint32_t)(a >> 32) * 4.656612873077393e-10f, &sn, &cs);  // x 2^-31: half turns
      to[k] = make_float2(cs, sn);
    }
    __syncthreads();
  }
  int slot = -1;
  if (PAGED) {
    slot = there ? __ldcg(p.slots + row) : -1;
    if (slot != -1 && (slot < 0 || (slot >> p.L.pshift) >= p.L.npages)) {
      if (c == 0) set_status(p.status, FT_DEV_RANGE);
      slot = -1;
    }
  }
  int hh = h0;
  // the heads up to `end`, all of one kind, each read while the one before it is worked on
  auto heads = [&](int end, const float* gamma, bool rotated, bool wide, auto&& put) {
    if (hh >= end) return;
    // z_lo = lo (g_lo cos) - hi (g_hi sin), z_hi = hi (g_hi cos) + lo (g_lo sin), the gains inside the factors
    f32x2 lc[4], ls[4], hc[4], hs[4];
    if (rotated) {
      const float4* from = reinterpret_cast<const float4*>(&angles[lane / LV][8 * c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = from[i];  // cos, sin; cos, sin
        float lo[2] = {1.0f, 1.0f}, hi[2] = {1.0f, 1.0f};
        if (gamma) {
#pragma unroll
          for (int k = 0; k < 2; ++k) lo[k] = gamma[8 * c + 2 * i + k], hi[k] = gamma[D / 2 + 8 * c + 2 * i + k];
        }
        lc[i] = f32x2(lo[0] * a.x, lo[1] * a.z), ls[i] = f32x2(lo[0] * a.y, lo[1] * a.w);
        hc[i] = f32x2(hi[0] * a.x, hi[1] * a.z), hs[i] = f32x2(-hi[0] * a.y, -hi[1] * a.w);
      }
    }
    for (; hh < end; ++hh) {
      f32x2 x[8];
      rope_values(raw, x);
      if (hh + 1 < end) {
        src += D;
        rope_load<D>(src, wide, raw);
      } else if (hh + 1 < h1) {
        src = source(hh + 1);
        rope_load<D>(src, wide_of(hh + 1), raw);
      }
      if (gamma) {
        f32x2 ss[2] = {mul2(x[0], x[0]), mul2(x[4], x[4])};
#pragma unroll
        for (int i = 1; i < 4; ++i) ss[0] = fma2(x[i], x[i], ss[0]), ss[1] = fma2(x[4 + i], x[4 + i], ss[1]);
        float a, b;
        add2(ss[0], ss[1]).get(a, b);
        a += b;
#pragma unroll
        for (int o = 1; o < LV; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        const float r = rsqrtf(fmaf(a, 1.0f / D, p.eps));
        const f32x2 r2(r, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], r2);
      }
      if (rotated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 lo = x[i], hi = x[i + 4];
          x[i] = fma2(hi, hs[i], mul2(lo, lc[i]));
          x[i + 4] = fma2(lo, ls[i], mul2(hi, hc[i]));
        }
      }
      put(x);
    }
  };
  auto out = [&](uint16_t* base, int64_t stride, int first, int bit) {  // puts rows to BF16 rows, from this warp's first head on
    return [=, to = base + row * stride + (int64_t)(max(h0, first) - first) * D + 8 * c, wide = (p.wide & bit) != 0](const f32x2 (&x)[8]) mutable {
      if (there) rope_store<D>(to, wide, x);
      to += D;
    };
  };
  heads(min(h1, p.nq), p.gamma_q, true, (p.wide & kWideQ) != 0, out(p.q_out, p.q_out_stride, 0, kWideQOut));
  if constexpr (PAGED) {
    heads(min(h1, turned), p.gamma_k, true, (p.wide & kWideK) != 0, [&](f32x2 (&x)[8]) { rope_place<D>(p, x, false, hh - p.nq, slot); });
    heads(h1, nullptr, false, (p.wide & kWideV) != 0, [&](f32x2 (&x)[8]) { rope_place<D>(p, x, true, hh - turned, slot); });
  } else {
    heads(min(h1, turned), p.gamma_k, true, (p.wide & kWideK) != 0, out(p.k_out, p.k_out_stride, p.nq, kWideKOut));
  }
}

static int launch_rope(const ft_block_cfg& c, RopeRows& p, bool paged, cudaStream_t st) {
  p.nq = p.q ? c.n_q : 0;
  p.nkv = p.k ? c.n_kv : 0;
  p.heads = p.nq + p.nkv * (paged ? 2 : 1);
  p.eps = c.rms_eps;
  auto wide = [](const void* at, int64_t stride, int bit) { return ft_host::aligned16(at) && stride % 8 == 0 ? bit : 0; };
  p.wide = wide(p.q, p.q_stride, kWideQ) | wide(p.k, p.k_stride, kWideK) | wide(p.v, p.v_stride, kWideV) |
           wide(p.q_out, p.q_out_stride, kWideQOut) | wide(p.k_out, p.k_out_stride, kWideKOut);
  rope_turns(c.rope_base, c.head_dim, p.turn);
  const int rows = 512 / c.head_dim;
  const int64_t groups = ((int64_t)p.total + rows - 1) / rows;
  constexpr int W = kRopeThreads / 32;
  // Heads of a warp: as many as leave every SM 48 warps, the warps' shares equal.  24 / 48 / 96 warps (us): 2048 tokens'
  // rows 10.3 / 12.6 / 17.7, placement with reading back 24.8 / 23.7 / 29.6; 17k and 9k tokens alike.
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  const int most = (int)std::min<int64_t>(kRopeHeads, std::max<int64_t>(1, groups * p.heads / ((int64_t)sms * 48)));
  const int chunks = (p.heads + W * most - 1) / (W * most);
  p.per = (p.heads + W * chunks - 1) / (W * chunks);
  const int64_t blocks = groups * ((p.heads + W * p.per - 1) / (W * p.per));
  if (blocks > INT32_MAX) return FT_ERR_UNSUPPORTED;
  const auto kernel = c.head_dim == 128 ? (paged ? rope_rows_kernel<128, true> : rope_rows_kernel<128, false>)
                                        : (paged ? rope_rows_kernel<64, true> : rope_rows_kernel<64, false>);
  return launch_served(kernel, dim3((unsigned)blocks), dim3(kRopeThreads), 0, st, 1, p) == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // namespace ft

extern "C" {

int ft_qk_norm_rope_bf16(const ft_block_cfg* c, const uint16_t* q_bf16, int64_t q_stride, const uint16_t* k_bf16,
                         int64_t k_stride, const float* gamma_q, const float* gamma_k, const int32_t* positions, int total,
                         uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride, ft_stream stream) {
  const int st = ft_host::check_cfg(c);
  if (st != FT_OK) return st;
  if (total < 0 || (!q_bf16 && !k_bf16) || !q_bf16 != !q_out || !k_bf16 != !k_out) return FT_ERR_INVALID_ARG;
  const int64_t row_q = (int64_t)c->n_q * c->head_dim, row_k = (int64_t)c->n_kv * c->head_dim;
  if (q_bf16 && (q_stride < row_q || q_out_stride < row_q)) return FT_ERR_INVALID_ARG;
  if (k_bf16 && (k_stride < row_k || k_out_stride < row_k)) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  if (!positions) return FT_ERR_INVALID_ARG;
  ft::RopeRows p = {};
  p.q = q_bf16, p.k = k_bf16;
  p.q_out = q_out, p.k_out = k_out;
  p.q_stride = q_stride, p.k_stride = k_stride;
  p.q_out_stride = q_out_stride, p.k_out_stride = k_out_stride;
  p.gamma_q = gamma_q, p.gamma_k = gamma_k;
  p.pos = positions;
  p.total = total;
  return ft::launch_rope(*c, p, false, (cudaStream_t)stream);
}

int ft_kv_append_rope_paged_int4(const ft_block_cfg* c, void* pages, int n_pages, int page_size, const uint16_t* k_bf16,
                                 int64_t k_stride, const uint16_t* v_bf16, int64_t v_stride, const float* gamma_k,
                                 const int32_t* positions, const int32_t* slots, int total, const uint16_t* q_bf16,
                                 int64_t q_stride, const float* gamma_q, uint16_t* q_out, int64_t q_out_stride,
                                 int32_t* dev_status, ft_stream stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (total < 0 || !q_bf16 != !q_out) return FT_ERR_INVALID_ARG;
  const int64_t row_q = (int64_t)c->n_q * c->head_dim, row_k = (int64_t)c->n_kv * c->head_dim;
  if (q_bf16 && (q_stride < row_q || q_out_stride < row_q)) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  if (!k_bf16 || !v_bf16 || !positions || !slots || k_stride < row_k || v_stride < row_k) return FT_ERR_INVALID_ARG;
  ft::RopeRows p = {};
  p.q = q_bf16, p.k = k_bf16, p.v = v_bf16;
  p.q_out = q_out;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.gamma_q = gamma_q, p.gamma_k = gamma_k;
  p.pos = positions, p.slots = slots;
  p.pages = static_cast<uint8_t*>(pages);
  p.L = ft::paged_layout(*c, n_pages, page_size);
  p.total = total;
  p.hb = c->had_block;
  p.norm = ft::paged_norm(c->had_block);
  p.status = dev_status;
  return ft::launch_rope(*c, p, true, (cudaStream_t)stream);
}

}  // extern "C"
