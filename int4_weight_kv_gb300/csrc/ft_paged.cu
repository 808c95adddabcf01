// Paged 4-bit KV cache: block tables and slot maps from request lengths, placement
// of new K/V rows through a slot map, and reading rows back.
#include <algorithm>

#include "ft_paged.cuh"

namespace ft {

// ------------------------------------------------------------------ page map
// One launch (a decode step's call is bound by its latency).  Every CTA scans all request
// lengths for itself (B <= 8192: a few loads a thread), keeping the prefix sums of rows and
// of pages taken in shared memory, and the CTAs share the new table entries and the slots,
// four consecutive ones per binary search.  Where outputs alias the inputs that they advance
// (kv_len = ctx_len, free_head_out = free_head) the CTAs are one cluster of up to kMapCtas,
// which meets once after everyone has read them.  Measured (256 prompts, 260k rows): 31 us for
// one search a slot by eight CTAs, 5 us so; 50 us where lengths and head are advanced in place, by eight
// CTAs (32 requests of one token: 0.3 us more than 4.9).
constexpr int kMapCtas = 8, kMapThreads = 256, kMapMaxB = 8192, kMapRun = 4;

struct MapParams {
  const int32_t *ctx, *add, *free_pages, *free_head;
  int32_t *table, *head_out, *cu, *kv_len, *slots, *status;
  int B, stride, n_free, n_slots, n_pages, pshift, clustered;
};

constexpr int kMapWarps = kMapThreads / 32;

// Exclusive scans of two values per thread over the CTA, and their totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& total_a, long long& total_b,
                                            long long (*sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += ua, ib += ub;
  }
  if (lane == 31) sums[warp][0] = ia, sums[warp][1] = ib;
  __syncthreads();
  long long ba = 0, bb = 0;
  total_a = total_b = 0;
#pragma unroll
  for (int w = 0; w < kMapWarps; ++w) {
    if (w == warp) ba = total_a, bb = total_b;
    total_a += sums[w][0];
    total_b += sums[w][1];
  }
  a = ba + ia - a;
  b = bb + ib - b;
}

// Largest i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const MapParams p) {
  extern __shared__ int32_t map_smem[];
  __shared__ long long sums[kMapWarps][2];
  __shared__ int bad, most;
  griddep_serve();
  const int tid = threadIdx.x, B = p.B;
  int32_t* cu = map_smem;       // [B + 1] first row of each request
  int32_t* pg = cu + B + 1;     // [B + 1] first page taken by each request
  int32_t* ctx_s = pg + B + 1;  // [B] history length, -1: not served
  const int per = (B + kMapThreads - 1) / kMapThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  const long long cap = min((long long)p.stride << p.pshift, (long long)INT32_MAX);  // positions of one table row
  const int round = (1 << p.pshift) - 1;
  // pages that c + a positions need beyond those of c; -1: not within a table row
  auto pages_added = [&](int c, int a) -> long long {
    if (c < 0 || a < 0 || (long long)c + a > cap) return -1;
    return (((long long)c + a + round) >> p.pshift) - (((long long)c + round) >> p.pshift);
  };
  const int head = p.free_head ? *p.free_head : 0;
  int c0 = 0, a0 = 0;  // the thread's first request (its only one up to B = 256), read once
  if (b0 < b1) c0 = p.ctx[b0], a0 = p.add[b0];
  if (tid == 0) bad = most = 0;
  long long r = 0, q = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = b == b0 ? c0 : p.ctx[b], a = b == b0 ? a0 : p.add[b];
    r += max(a, 0);
    q += max(pages_added(c, a), 0ll);
  }
  long long n_rows, n_need;
  block_scan2(r, q, n_rows, n_need, sums);
  const long long avail = (head >= 0 && head <= p.n_free) ? p.n_free - head : 0;
  for (int b = b0; b < b1; ++b) {
    const int c = b == b0 ? c0 : p.ctx[b], a = b == b0 ? a0 : p.add[b];
    cu[b] = (int)min(r, (long long)INT32_MAX);
    pg[b] = (int)min(q, (long long)INT32_MAX);
    r += max(a, 0);
    const long long n = pages_added(c, a);
    bool served = n >= 0;
    if (n > 0) {
      q += n;
      served = q <= avail;
      if (served) atomicMax(&most, (int)q);  // pages taken: the largest prefix sum that a served request reached
    }
    ctx_s[b] = served ? c : -1;
    if (!served) bad = FT_DEV_CAPACITY;  // the same value from every thread
  }
  if (tid == 0) {
    cu[B] = (int)min(n_rows, (long long)INT32_MAX);
    pg[B] = (int)min(n_need, (long long)INT32_MAX);
  }
  if (p.clustered) {
    cluster_arrive();
    cluster_wait();  // every CTA has read the lengths and the head
  } else {
    __syncthreads();
  }
  const int n_taken = most, total = min(cu[B], p.n_slots);
  const int first = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
  if (blockIdx.x == 0) {
    for (int b = tid; b <= B; b += kMapThreads) p.cu[b] = cu[b];
    for (int b = tid; b < B; b += kMapThreads)  // (not from cu, whose sums end at 2^31 - 1)
      p.kv_len[b] = ctx_s[b] < 0 ? 0 : ctx_s[b] + (b == b0 ? a0 : p.add[b]);
    if (tid == 0) {
      if (p.head_out) *p.head_out = head + n_taken;
      int flags = bad;
      if (n_rows > p.n_slots || head < 0 || head > p.n_free) flags |= FT_DEV_RANGE;
      if (flags) set_status(p.status, flags);
    }
  }
  // page id of the free list's entry i, or -1 (and a flag) where it is no page
  auto fresh = [&](int64_t i) {
    const int id = p.free_pages[head + i];
    if (id >= 0 && id < p.n_pages) return id;
    set_status(p.status, FT_DEV_RANGE);
    return -1;
  };
  // (indices of 64 bits: a step behind the last entry would pass 2^31 where there are nearly that many)
  for (int64_t i = first; i < n_taken; i += step) {
    const int b = last_not_above(pg, B, (int)i);
    const int old = (int)(((long long)ctx_s[b] + round) >> p.pshift);
    if (ctx_s[b] >= 0) p.table[(size_t)b * p.stride + old + (i - pg[b])] = fresh(i);
  }
  for (int64_t i0 = kMapRun * first; i0 < p.n_slots; i0 += kMapRun * step) {
    int out[kMapRun], b = 0, last_ip = -1, id = -1;
    if (i0 < total) b = last_not_above(cu, B, (int)i0);
#pragma unroll
    for (int k = 0; k < kMapRun; ++k) {
      const int64_t i = i0 + k;
      out[k] = -1;
      if (i >= total) continue;
      if (i >= cu[b + 1]) {
        do ++b;
        while (i >= cu[b + 1]);
        last_ip = -1;
      }
      const int c = ctx_s[b];
      if (c < 0) continue;
      const int pos = c + ((int)i - cu[b]), ip = pos >> p.pshift;
      if (ip != last_ip) {
        const int old = (int)(((long long)c + round) >> p.pshift);
        id = ip < old ? p.table[(size_t)b * p.stride + ip] : fresh(pg[b] + ip - old);
        if (id < 0 || id >= p.n_pages) {
          set_status(p.status, FT_DEV_RANGE);
          id = -1;
        }
        last_ip = ip;
      }
      if (id >= 0) out[k] = (id << p.pshift) + (pos & round);
    }
    if (i0 + kMapRun <= p.n_slots && (reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0) {
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kMapRun; ++k)
        if (i0 + k < p.n_slots) p.slots[i0 + k] = out[k];
    }
  }
}

// ------------------------------------------------------------------ placement
// D / 32 lanes per row of one head, K (blockIdx.y 0) or V; a warp holds 32 / (D / 32)
// consecutive rows of one head, so that a prompt's entries leave it as contiguous pieces
// and the two positions of a V pair meet in neighbouring groups of lanes.  The rotated row
// is quantised in the registers where it was formed: no shared memory.  Bound by the issue slots
// (450 warp instructions for eight rows, 380 to read back; 72% of the slots used): 16384 tokens of 8
// heads of 128, K and V, 26 us and 24 us, 3.3 and 3.6 TB/s.
constexpr int kRowThreads = 128;

struct PagedRows {
  const uint16_t *k, *v;
  uint16_t *k_out, *v_out;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  uint8_t* pages;
  PagedLayout L;
  int total, hb;
  float norm;
  int32_t* status;
};

// This thread's row: t (total: none), head, lane of the row and its slot as given.
template <int D>
__device__ __forceinline__ void paged_row(const PagedRows& p, int& t, int& h, int& j, int& slot) {
  constexpr int LV = D / 32, R = 32 / LV;  // lanes of a row, rows of a warp
  const int64_t warp = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  h = (int)(warp % p.L.nkv);
  const int64_t row = (warp / p.L.nkv) * R + lane / LV;
  t = (int)min(row, (int64_t)p.total);
  j = lane % LV;
  slot = t < p.total ? __ldcg(p.slots + t) : -1;
}
// The slot, or -1 (and a flag) where it is none.
__device__ __forceinline__ int paged_slot(const PagedRows& p, int slot, int j) {
  if (slot == -1 || (slot >= 0 && (slot >> p.L.pshift) < p.L.npages)) return slot;
  if (j == 0) set_status(p.status, FT_DEV_RANGE);
  return -1;
}

// NaN where either is, else the larger.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kMagic = 12582912.0f;  // 1.5 2^23: |x| r + kMagic rounds to the nearest integer, ties to even

// Codes of words g and g + 1 (values u[e][0] and u[e][1], as kMagic + magnitude; x the signed
// values) as one register: magnitudes at bits 0, 3, 8, 11, signs at bits 15, 14, 7, 6 of each half.
__device__ __forceinline__ uint32_t paged_pack(const f32x2 (&x)[4], const f32x2 (&u)[4]) {
  constexpr uint32_t kTop = 0x4B400000u, kAll = (1u + (1u << 3) + (1u << 8) + (1u << 11)) * kTop;
  uint32_t xs[4][2], w = 0u - kAll - (kAll << 16);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    u[e].get(a, b);
    const int at = (e & 1) * 3 + (e >> 1) * 8;
    w += (__float_as_uint(a) << at) + (__float_as_uint(b) << (at + 16));
    x[e].get(a, b);
    xs[e][0] = __float_as_uint(a), xs[e][1] = __float_as_uint(b);
  }
  // sign bytes: (value 0, value 2) and (value 1, value 3) as the halves' high and low bytes
  const uint32_t s02 = prmt(prmt(xs[2][0], xs[0][0], 0x0073u), prmt(xs[2][1], xs[0][1], 0x0073u), 0x5410u);
  const uint32_t s13 = prmt(prmt(xs[3][0], xs[1][0], 0x0073u), prmt(xs[3][1], xs[1][1], 0x0073u), 0x5410u);
  return w | (s02 & 0x80808080u) | ((s13 >> 1) & 0x40404040u);
}

// Magnitude of the code of y = fl(|x| norm) by scale s, min(rne(fl(y / s)), 7), decided without a
// division where c = rne(y / s) is right but perhaps for the side of a boundary.  With t the
// nearest boundary, y - t s is exact; the FP32 quotient is t itself (and the even neighbour its
// code) while that is within half a step of t, else its sign decides.
__device__ __noinline__ float paged_edge(float y, float s, float c) {
  if (!(s >= 1e-30f)) return s > 0.0f ? fminf(rintf(__fdiv_rn(y, s)), 7.0f) : 0.0f;
  const float t = fmaf(-c, s, y) > 0.0f ? c + 0.5f : c - 0.5f, rem = fmaf(-t, s, y);
  const float step = __uint_as_float((__float_as_uint(t) & 0x7F800000u) - (24u << 23));  // half a step above t
  const float half = (rem < 0.0f && t == 0.5f) ? 0.5f * step : step;                     // below a power of two: half of it
  const float lo = t - 0.5f, hi = t + 0.5f;
  if (fabsf(rem) <= s * half) return ((int)lo & 1) ? hi : lo;
  return fminf(rem > 0.0f ? hi : lo, 7.0f);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) append_paged_kernel(const PagedRows p) {
  constexpr int LV = D / 32;
  griddep_serve();
  int t, h, j, slot;
  paged_row<D>(p, t, h, j, slot);
  const bool is_v = blockIdx.y != 0;
  f32x2 x[16];
  if (t < p.total) {
    const uint16_t* src = (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * D + 32 * j;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(src)[i];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[4 * i + k] = f32x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = f32x2(bf16_bits_to_f32(src[2 * i]), bf16_bits_to_f32(src[2 * i + 1]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = f32x2(0.0f, 0.0f);
  }
  slot = paged_slot(p, slot, j);  // after the row's loads: its own load is under way beside them
  paged_fwht<D>(x, p.hb);
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    x[i].get(a, b);
    am = max_nan(am, max_nan(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = 1; o < LV; o <<= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  const bool finite = am < INFINITY;
  const uint16_t sb = quant_scale_bits(am * p.norm);
  const float s = bf16_bits_to_f32(sb);
  // Codes by a reciprocal: |x| (norm r) is within 2^-22 (relative) of the quotient fl(x norm) / s
  // rounded to FP32 that the quantiser takes its decision from, so the two agree unless it lies
  // within 7 x 2^-21 of a rounding boundary; those few values are decided exactly.
  const float r = s >= 1e-30f ? p.norm * __frcp_rn(s) : 0.0f;
  const f32x2 r2(r, r), magic2(kMagic, kMagic), minus(-1.0f, -1.0f);
  const float far = r > 0.0f || s == 0.0f ? 0.5f - 7.0f * 4.76837158203125e-07f : -1.0f;  // 7 x 2^-21
  uint32_t hw[4];  // words 2 q and 2 q + 1 of this lane's 32 channels
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f32x2 xe[4], u[4];
    float near = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      xe[e] = x[4 * e + q];
      xe[e].get(a, b);
      const f32x2 mag(fabsf(a), fabsf(b));
      u[e] = fma2(mag, r2, magic2);
      fma2(mag, r2, fma2(u[e], minus, magic2)).get(a, b);
      near = fmaxf(near, fmaxf(fabsf(a), fabsf(b)));
    }
    if (near >= far) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[2], m[2];
        xe[e].get(v[0], v[1]);
        u[e].get(m[0], m[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = fabsf(v[i]), c = m[i] - kMagic;
          if (fabsf(fmaf(a, r, -c)) >= far) m[i] = kMagic + paged_edge(a * p.norm, s, c);
        }
        u[e] = f32x2(m[0], m[1]);
      }
    }
    hw[q] = paged_pack(xe, u);
  }
  // a NaN's "code" may spill over its neighbours' bits: such a row is not defined, only flagged
  if (!finite && slot >= 0) set_status(p.status, FT_DEV_RANGE);
  const int pos = max(slot, 0) & (p.L.psize - 1);
  uint8_t* blk = p.pages + paged_block(p.L, max(slot, 0) >> p.L.pshift, h);
  if (!is_v) {
    if (slot >= 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint32_t*>(blk + paged_k_word<D>(pos, 2 * q, j)) = hw[q];
    }
  } else {
    // the pair's other position in the neighbouring lanes: each side stores four whole words
    const int other = __shfl_xor_sync(0xffffffffu, slot, LV);
    const bool pair = slot >= 0 && other == (slot ^ 1);
    const bool odd = (slot & 1) != 0;
    uint32_t got[2], keep[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      got[q] = __shfl_xor_sync(0xffffffffu, odd ? hw[q] : hw[2 + q], LV);
      keep[q] = odd ? hw[2 + q] : hw[q];
    }
    uint8_t* dst = blk + p.L.voff;
    if (pair) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t even_w = odd ? got[q] : keep[q], odd_w = odd ? keep[q] : got[q];
        const int g = (odd ? 4 : 0) + 2 * q;
        *reinterpret_cast<uint32_t*>(dst + paged_v_word<D>(pos & ~1, g, j)) = prmt(even_w, odd_w, 0x5410u);
        *reinterpret_cast<uint32_t*>(dst + paged_v_word<D>(pos & ~1, g + 1, j)) = prmt(even_w, odd_w, 0x7632u);
      }
    } else if (slot >= 0) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        *reinterpret_cast<uint16_t*>(dst + paged_v_word<D>(pos, g, j)) = (uint16_t)(hw[g / 2] >> (16 * (g & 1)));
    }
  }
  if (slot >= 0 && j == 0) *reinterpret_cast<uint16_t*>(blk + p.L.soff + 4 * pos + (is_v ? 2 : 0)) = sb;
}

// Rows of the given slots as values in the model basis: decoded, rotated back,
// rounded to BF16.  (Nine CTAs an SM: left alone the compiler takes 62 registers, 0.2 us more for 16384 tokens.)
template <int D>
__global__ void __launch_bounds__(kRowThreads, 9) read_paged_kernel(const PagedRows p) {
  griddep_serve();
  int t, h, j, slot;
  paged_row<D>(p, t, h, j, slot);
  slot = paged_slot(p, slot, j);
  const bool is_v = blockIdx.y != 0;
  const int pos = max(slot, 0) & (p.L.psize - 1);
  const uint8_t* blk = p.pages + paged_block(p.L, max(slot, 0) >> p.L.pshift, h);
  uint32_t w[4] = {0u, 0u, 0u, 0u};  // words 2 q, 2 q + 1
  float s = 0.0f;
  if (slot >= 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (is_v) {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(blk + p.L.voff + paged_v_word<D>(pos & ~1, 2 * q, j));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(blk + p.L.voff + paged_v_word<D>(pos & ~1, 2 * q + 1, j));
        w[q] = prmt(a, b, (pos & 1) ? 0x7632u : 0x5410u);
      } else {
        w[q] = *reinterpret_cast<const uint32_t*>(blk + paged_k_word<D>(pos, 2 * q, j));
      }
    }
    const uint32_t both = *reinterpret_cast<const uint32_t*>(blk + p.L.soff + 4 * pos);
    s = __uint_as_float(is_v ? both & 0xFFFF0000u : both << 16);
  }
  // The decoded halves are x 2^-24 (e even) and x 2^-20: made up for with the scale, or with the rotation's
  // factor where the scale is large (x 2^24 a scale passes FP32 from 2^104 on).
  const bool late = s >= 1.0f;
  const float up = late ? s : s * 16777216.0f;
  const f32x2 s0(up, up), s1(up * 0.0625f, up * 0.0625f);
  f32x2 x[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t r[4];
    paged_word(w[q], r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[e]));
      x[4 * e + q] = mul2(f32x2(f.x, f.y), (e & 1) ? s1 : s0);
    }
  }
  paged_fwht<D>(x, p.hb);
  if (t >= p.total) return;
  const float last = late ? p.norm * 16777216.0f : p.norm;
  const f32x2 norm2(last, last);
  uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((int64_t)t * p.L.nkv + h) * D + 32 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      mul2(x[4 * i + k], norm2).get(a, b);
      const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
      o[k] = *reinterpret_cast<const uint32_t*>(&r);
    }
    dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Grid over (rows, heads) x (K, V); 0 blocks: too many.
static dim3 row_grid(int total, int nkv, int d) {
  const int per = 32 / (d / 32);
  const int64_t warps = ((int64_t)total + per - 1) / per * nkv, blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  return dim3(blocks > INT32_MAX ? 0u : (unsigned)blocks, 2);
}

}  // namespace ft

extern "C" {

size_t ft_kv_pages_bytes(const ft_block_cfg* c, int n_pages, int page_size) {
  if (ft_host::check_cfg(c) != FT_OK || !ft::paged_size_ok(page_size)) return 0;
  if (n_pages < 1 || n_pages > INT32_MAX / page_size) return 0;
  return (size_t)n_pages * c->n_kv * ft::paged_layout(*c, n_pages, page_size).block;
}

int ft_kv_page_map(int page_size, int n_pages, const int32_t* ctx_len, const int32_t* new_len, int B,
                   int32_t* block_table, int table_stride, const int32_t* free_pages, int n_free,
                   const int32_t* free_head, int32_t* free_head_out, int32_t* cu_seqlens, int32_t* kv_len,
                   int32_t* slots, int n_slots, int32_t* dev_status, ft_stream stream) {
  if (!ft::paged_size_ok(page_size)) return FT_ERR_UNSUPPORTED;
  if (n_pages < 1 || n_pages > INT32_MAX / page_size) return FT_ERR_INVALID_ARG;
  if (!ctx_len || !new_len || !block_table || !cu_seqlens || !kv_len || B < 1 || table_stride < 1 || n_free < 0 ||
      n_slots < 0 || (n_free > 0 && !free_pages) || (n_slots > 0 && !slots))
    return FT_ERR_INVALID_ARG;
  if (B > ft::kMapMaxB) return FT_ERR_UNSUPPORTED;
  ft::MapParams p = {};
  p.ctx = ctx_len;
  p.add = new_len;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.table = block_table;
  p.head_out = free_head_out;
  p.cu = cu_seqlens;
  p.kv_len = kv_len;
  p.slots = slots;
  p.status = dev_status;
  p.B = B;
  p.stride = table_stride;
  p.n_free = n_free;
  p.n_slots = n_slots;
  p.n_pages = n_pages;
  p.pshift = 31 - __builtin_clz((unsigned)page_size);
  const int smem = (3 * B + 2) * 4;
  static int attr_smem[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FT_ERR_CUDA;
  // (without the attribute 48 KB hold the kernel's static variables too)
  if (smem > 48 * 1024 - 1024 && attr_smem[dev] < smem) {
    const int most = (3 * ft::kMapMaxB + 2) * 4;
    if (cudaFuncSetAttribute(ft::page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return FT_ERR_CUDA;
    attr_smem[dev] = most;
  }
  // a CTA for every 1024 rows; one cluster where an output is also an input
  p.clustered = kv_len == ctx_len || (free_head_out && free_head_out == free_head) ? 1 : 0;
  const int want = (int)(((int64_t)n_slots + ft::kMapRun * ft::kMapThreads - 1) / (ft::kMapRun * ft::kMapThreads));
  int ctas = 1;
  if (p.clustered) {
    while (ctas < ft::kMapCtas && ctas < want) ctas *= 2;
  } else {
    const int sms = ft_host::num_sms();
    ctas = std::max(1, std::min(want, 2 * (sms > 0 ? sms : 152)));
  }
  return ft::launch_served(ft::page_map_kernel, dim3(ctas), dim3(ft::kMapThreads), smem, (cudaStream_t)stream,
                           p.clustered ? ctas : 1, p) == cudaSuccess
             ? FT_OK
             : FT_ERR_CUDA;
}

int ft_kv_append_paged_int4(const ft_block_cfg* c, void* pages, int n_pages, int page_size, const uint16_t* k_bf16,
                            int64_t k_stride, const uint16_t* v_bf16, int64_t v_stride, const int32_t* slots, int total,
                            int32_t* dev_status, ft_stream stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (total < 0) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  const int64_t row = (int64_t)c->n_kv * c->head_dim;
  if (!k_bf16 || !v_bf16 || !slots || k_stride < row || v_stride < row) return FT_ERR_INVALID_ARG;
  ft::PagedRows p = {};
  p.k = k_bf16;
  p.v = v_bf16;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.pages = static_cast<uint8_t*>(pages);
  p.L = ft::paged_layout(*c, n_pages, page_size);
  p.total = total;
  p.hb = c->had_block;
  p.norm = ft::paged_norm(c->had_block);
  p.status = dev_status;
  const dim3 grid = ft::row_grid(total, c->n_kv, c->head_dim);
  if (grid.x == 0) return FT_ERR_UNSUPPORTED;
  const auto kernel = c->head_dim == 128 ? ft::append_paged_kernel<128> : ft::append_paged_kernel<64>;
  return ft::launch_served(kernel, grid, dim3(ft::kRowThreads), 0, (cudaStream_t)stream, 1, p) == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

int ft_kv_read_paged_int4(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const int32_t* slots,
                          int total, uint16_t* k_out, uint16_t* v_out, int32_t* dev_status, ft_stream stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (total < 0) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  if (!slots || !k_out || !v_out || !ft_host::aligned16(k_out) || !ft_host::aligned16(v_out)) return FT_ERR_INVALID_ARG;
  ft::PagedRows p = {};
  p.k_out = k_out;
  p.v_out = v_out;
  p.slots = slots;
  p.pages = static_cast<uint8_t*>(const_cast<void*>(pages));
  p.L = ft::paged_layout(*c, n_pages, page_size);
  p.total = total;
  p.hb = c->had_block;
  p.norm = ft::paged_norm(c->had_block);
  p.status = dev_status;
  const dim3 grid = ft::row_grid(total, c->n_kv, c->head_dim);
  if (grid.x == 0) return FT_ERR_UNSUPPORTED;
  const auto kernel = c->head_dim == 128 ? ft::read_paged_kernel<128> : ft::read_paged_kernel<64>;
  return ft::launch_served(kernel, grid, dim3(ft::kRowThreads), 0, (cudaStream_t)stream, 1, p) == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
