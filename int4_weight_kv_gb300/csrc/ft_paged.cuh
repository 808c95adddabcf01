// Layout of the paged 4-bit KV cache and the device helpers shared by its
// kernels (placement, reading back, attention).
//
// A page holds page_size positions of every KV head: n_kv head blocks of
// page_size (d + 4) bytes, each
//   K     page_size entries of d/2 bytes
//   V     page_size / 2 pair entries of d bytes (positions 2i and 2i + 1)
//   scale page_size x (BF16 K scale, BF16 V scale)
// so that one (page, head) is one contiguous piece, a multiple of 16 bytes.
//
// Values are sign and magnitude, four per 16-bit word.  Word (g, j) of a
// position holds channels 32 j + g + 8 e as value e = 0..3: magnitudes (0..7) at
// bits 0, 3, 8, 11 and signs at bits 15, 14, 7, 6.  Masked (after a shift left by
// one for e = 1 and 3, on the byte-swapped word for e = 2 and 3), a value is an
// FP16 subnormal: sign x magnitude x 2^-24, and 16 times that for odd e (channels
// with c % 16 >= 8).  The tensor cores take subnormals exactly, so four values of
// two words decode in seven integer instructions with no offset to subtract
// afterwards (an offset code's 8 sum P would cancel against the result, and its
// truncation bias grows with the context).
//   K: 32-bit words join the channel pair g = 2t, 2t + 1: chunk t (d/8 bytes) holds
//      words j = 0..d/32-1 of lane column t, the A fragment of two k-steps a word.
//   V: 32-bit words join positions 2i (low half) and 2i + 1: chunk g (d/8 bytes)
//      of a pair holds words j of channels == g mod 8, stored at chunk
//      g ^ paged_v_turn(i), which keeps 16-byte (8-byte, d = 64) shared-memory
//      reads of four pairs by eight lanes on different banks.
#pragma once

#include <cmath>

#include "ft_internal.cuh"

namespace ft {

struct PagedLayout {
  int nkv, npages, psize, pshift;  // positions per page = 1 << pshift
  uint32_t voff, soff, block;      // V and scale offsets in a head block, its bytes
};

inline bool paged_size_ok(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

inline PagedLayout paged_layout(const ft_block_cfg& c, int n_pages, int page_size) {
  PagedLayout L;
  L.nkv = c.n_kv;
  L.npages = n_pages;
  L.psize = page_size;
  L.pshift = 31 - __builtin_clz((unsigned)page_size);
  L.voff = (uint32_t)page_size * c.head_dim / 2;
  L.soff = (uint32_t)page_size * c.head_dim;
  L.block = (uint32_t)page_size * (c.head_dim + 4);
  return L;
}

// Head block of (page, KV head): 64-bit offsets, a pool passes 4 GiB easily.
__device__ __forceinline__ size_t paged_block(const PagedLayout& L, int page, int h) {
  return ((size_t)page * L.nkv + h) * L.block;
}

template <int D>
__host__ __device__ __forceinline__ int paged_v_turn(int pair) {
  return D == 128 ? 2 * (pair & 3) : 4 * ((pair >> 1) & 1);
}
// Byte offset of word (g, j) of position p (inside the page) in the K part, and in the V part.
template <int D>
__device__ __forceinline__ uint32_t paged_k_word(int p, int g, int j) {
  return (uint32_t)(p * (D / 2) + (g >> 1) * (D / 8) + 4 * j + 2 * (g & 1));
}
template <int D>
__device__ __forceinline__ uint32_t paged_v_word(int p, int g, int j) {
  return (uint32_t)((p >> 1) * D + (g ^ paged_v_turn<D>(p >> 1)) * (D / 8) + 4 * j + 2 * (p & 1));
}

// Two words' values as FP16 pairs: r[e] holds value e of the low and the high
// 16 bits, x 2^-24 (e even) or x 16 2^-24 (e odd).
__device__ __forceinline__ void paged_word(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t sw = prmt(w, 0u, 0x2301u);  // bytes of each half swapped
  r[0] = w & 0x80078007u;
  r[1] = (w << 1) & 0x80708070u;
  r[2] = sw & 0x80078007u;
  r[3] = (sw << 1) & 0x80708070u;
}
// Walsh-Hadamard transform (order hb, natural order, not yet normalised) of a d-vector
// held by D / 32 neighbouring lanes, lane j owning channels 32 j .. 32 j + 31: five
// strides inside a lane, the last two (one for d = 64) across lanes, so a vector costs 8
// shuffles of a warp where four channels a lane would cost 20.  Strides 1, 2, 4, ... in
// this order, FP32, so every lane layout and the plain form round alike.
// Channels 2 i and 2 i + 1 are pair i: one instruction adds two.
template <int D>
__device__ __forceinline__ void paged_fwht(f32x2 (&v)[16], int hb) {
  const f32x2 minus(-1.0f, -1.0f);
  if (hb > 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, b;
      v[i].get(a, b);
      v[i] = f32x2(a + b, a - b);
    }
  }
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) {
    if (2 * s >= hb) break;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i & s) continue;
      const f32x2 a = v[i], b = v[i + s];
      v[i] = add2(a, b);
      v[i + s] = fma2(b, minus, a);
    }
  }
#pragma unroll
  for (int s = 1; s < D / 32; s <<= 1) {
    if (32 * s >= hb) break;
    const float sign = (threadIdx.x & s) ? -1.0f : 1.0f;
    const f32x2 sign2(sign, sign);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, b;
      v[i].get(a, b);
      const f32x2 o(__shfl_xor_sync(0xffffffffu, a, s), __shfl_xor_sync(0xffffffffu, b, s));
      v[i] = fma2(sign2, v[i], o);
    }
  }
}

inline float paged_norm(int hb) { return (float)(1.0 / std::sqrt((double)hb)); }

}  // namespace ft

namespace ft_host {

// Checks shared by the calls on a paged cache.
inline int check_paged(const ft_block_cfg* c, const void* pages, int n_pages, int page_size) {
  const int st = check_cfg(c);
  if (st != FT_OK) return st;
  if (!ft::paged_size_ok(page_size)) return FT_ERR_UNSUPPORTED;
  if (n_pages < 1 || n_pages > INT32_MAX / page_size) return FT_ERR_INVALID_ARG;
  if (!pages || !aligned16(pages)) return FT_ERR_INVALID_ARG;
  return FT_OK;
}

}  // namespace ft_host
