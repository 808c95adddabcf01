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
// Value e of a 16-bit word as a float (an integer in -7..7).
__device__ __forceinline__ float paged_value(uint32_t w, int e) {
  const int mag = (w >> ((e & 1) * 3 + (e >> 1) * 8)) & 7;
  const int neg = (w >> (e == 0 ? 15 : e == 1 ? 14 : e == 2 ? 7 : 6)) & 1;
  return (float)(neg ? -mag : mag);
}
// 16-bit word of four codes in -7..7.
__device__ __forceinline__ uint32_t paged_pack(int c0, int c1, int c2, int c3) {
  uint32_t w = (uint32_t)abs(c0) | ((uint32_t)abs(c1) << 3) | ((uint32_t)abs(c2) << 8) | ((uint32_t)abs(c3) << 11);
  w |= (c0 < 0 ? 0x8000u : 0u) | (c1 < 0 ? 0x4000u : 0u) | (c2 < 0 ? 0x80u : 0u) | (c3 < 0 ? 0x40u : 0u);
  return w;
}

// Normalised Walsh-Hadamard transform (order hb, natural order) of a d-vector held
// by D / 4 neighbouring lanes: lane (g = channel bits 0-2, j = bits 5 and up) owns
// the four channels 32 j + g + 8 e.  Strides 1, 2, 4, ... in this order, FP32, so
// every lane layout and the plain form round alike.
template <int D>
__device__ __forceinline__ void paged_fwht(float (&v)[4], int hb, float norm) {
  const int lane = threadIdx.x & 31;
  auto across = [&](int s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float o = __shfl_xor_sync(0xffffffffu, v[e], s);
      v[e] = (lane & s) ? (o - v[e]) : (v[e] + o);
    }
  };
  if (hb > 1) across(1);
  if (hb > 2) across(2);
  if (hb > 4) across(4);
  if (hb > 8) {
    const float a = v[0], b = v[1], c = v[2], d = v[3];
    v[0] = a + b, v[1] = a - b, v[2] = c + d, v[3] = c - d;
  }
  if (hb > 16) {
    const float a = v[0], b = v[1], c = v[2], d = v[3];
    v[0] = a + c, v[2] = a - c, v[1] = b + d, v[3] = b - d;
  }
  if (hb > 32) across(8);
  if (D == 128 && hb > 64) across(16);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] *= norm;
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
