// Rows of the fused projection made ready for the cache and for attention: per-head RMS norms and the
// position rotation of q and k, and the placement of k and v in the paged 4-bit cache on the way.
//
//   y = gamma x / sqrt(mean x^2 + eps),   z_i = y_i cos a - y_(i+d/2) sin a,  z_(i+d/2) = y_(i+d/2) cos a + y_i sin a
#include <algorithm>

#include "ft_paged.cuh"

namespace ft {

// D / 16 lanes per row: lane c owns channels 8 c .. 8 c + 7 and d/2 + 8 c .. d/2 + 8 c + 7, two 16-byte
// pieces, so that the pairs of the rotation meet in one lane.  A warp holds 4 (8) consecutive tokens of one
// head and goes through `per` heads with the same angles.
constexpr int kRopeThreads = 128;

struct RopeRows {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const float *gamma_q, *gamma_k;
  const int32_t *pos, *slots;
  uint8_t* pages;
  PagedLayout L;
  int total, nq, nkv, heads, per, hb;  // heads: nq q heads, then k, then (paged) v; per: those of a warp
  float norm, eps;
  int32_t* status;
  uint64_t turn[64];
};

__device__ __forceinline__ void rope_load8(const uint16_t* src, f32x2* x) {
  if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
    const uint4 q = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x2(bf16_bits_to_f32(src[2 * i]), bf16_bits_to_f32(src[2 * i + 1]));
  }
}
__device__ __forceinline__ void rope_store8(uint16_t* dst, const f32x2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    x[i].get(a, b);
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[2 * i] = (uint16_t)w[i], dst[2 * i + 1] = (uint16_t)(w[i] >> 16);
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
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b, m0, m1, d0, d1;
    x[i].get(a, b);
    const f32x2 mag(fabsf(a), fabsf(b)), u = fma2(mag, r2, magic2);
    fma2(mag, r2, fma2(u, minus, magic2)).get(d0, d1);
    u.get(m0, m1);
    if (fmaxf(fabsf(d0), fabsf(d1)) >= far) {
      if (fabsf(d0) >= far) m0 = kMagic + paged_edge(fabsf(a) * p.norm, s, m0 - kMagic);
      if (fabsf(d1) >= far) m1 = kMagic + paged_edge(fabsf(b) * p.norm, s, m1 - kMagic);
    }
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

template <int D, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeRows p) {
  constexpr int LV = D / 16, R = 32 / LV;
  griddep_serve();
  const int lane = threadIdx.x & 31, c = lane % LV;
  const int chunks = (p.heads + p.per - 1) / p.per;
  const int64_t warp = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = warp / chunks * R + lane / LV;
  if (t - lane / LV >= p.total) return;
  const bool there = t < p.total;
  const int h0 = (int)(warp % chunks) * p.per, h1 = min(h0 + p.per, p.heads), turned = p.nq + p.nkv;
  int slot = -1;
  if (PAGED) {
    slot = there ? __ldcg(p.slots + t) : -1;
    if (slot != -1 && (slot < 0 || (slot >> p.L.pshift) >= p.L.npages)) {
      if (c == 0) set_status(p.status, FT_DEV_RANGE);
      slot = -1;
    }
  }
  f32x2 cs[4], sn[4];
  if (h0 < turned) {
    const int pos = there ? p.pos[t] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float c2[2], s2[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint64_t a = (uint64_t)(int64_t)pos * p.turn[8 * c + 2 * i + k];  // turns, modulo one
        sincospif((float)(int32_t)(uint32_t)(a >> 32) * 4.656612873077393e-10f, &s2[k], &c2[k]);  // x 2^-31: half turns
      }
      cs[i] = f32x2(c2[0], c2[1]);
      sn[i] = f32x2(s2[0], s2[1]);
    }
  }
  const f32x2 minus(-1.0f, -1.0f);
  for (int hh = h0; hh < h1; ++hh) {
    const int kind = hh < p.nq ? 0 : hh < turned ? 1 : 2, h = hh - (kind == 0 ? 0 : kind == 1 ? p.nq : turned);
    const uint16_t* src = (kind == 0 ? p.q + t * p.q_stride : kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride) + h * D + 8 * c;
    f32x2 x[8];
    if (there) {
      rope_load8(src, x);
      rope_load8(src + D / 2, x + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = f32x2(0.0f, 0.0f);
    }
    if (kind < 2) {
      const float* gamma = kind == 0 ? p.gamma_q : p.gamma_k;
      if (gamma) {
        f32x2 ss = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) ss = fma2(x[i], x[i], ss);
        float a, b;
        ss.get(a, b);
        a += b;
#pragma unroll
        for (int o = 1; o < LV; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        const float r = rsqrtf(fmaf(a, 1.0f / D, p.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int ch = (i < 4 ? 0 : D / 2) + 8 * c + 2 * (i & 3);
          x[i] = mul2(mul2(x[i], f32x2(r, r)), f32x2(gamma[ch], gamma[ch + 1]));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 lo = x[i], hi = x[i + 4];
        x[i] = fma2(mul2(hi, sn[i]), minus, mul2(lo, cs[i]));
        x[i + 4] = fma2(lo, sn[i], mul2(hi, cs[i]));
      }
    }
    if (PAGED && kind > 0) {
      rope_place<D>(p, x, kind == 2, h, slot);
    } else if (there) {
      uint16_t* dst = (kind == 0 ? p.q_out + t * p.q_out_stride : p.k_out + t * p.k_out_stride) + h * D + 8 * c;
      rope_store8(dst, x);
      rope_store8(dst + D / 2, x + 4);
    }
  }
}

static int launch_rope(const ft_block_cfg& c, RopeRows& p, bool paged, cudaStream_t st) {
  p.nq = p.q ? c.n_q : 0;
  p.nkv = p.k ? c.n_kv : 0;
  p.heads = p.nq + p.nkv * (paged ? 2 : 1);
  p.eps = c.rms_eps;
  rope_turns(c.rope_base, c.head_dim, p.turn);
  const int rows = 512 / c.head_dim;
  const int64_t groups = ((int64_t)p.total + rows - 1) / rows;
  p.per = (int)std::min<int64_t>(8, std::max<int64_t>(1, groups * p.heads / (152 * 48)));
  const int64_t warps = groups * ((p.heads + p.per - 1) / p.per), blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
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
