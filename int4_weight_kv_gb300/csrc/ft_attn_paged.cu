// Attention of any number of new tokens per request over the paged 4-bit cache.
//
// The formulas are at the top of ft_attn_paged.cuh.
#include <algorithm>

#include "ft_attn_paged.cuh"

namespace ft {

constexpr int kApWarps = 4;

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// ------------------------------------------------------------------ few rows
// Requests with up to 8 NT rows (tokens x heads of a group) a KV head: every byte of the
// cache is read once and used for all of them.  A 16-position tile costs a warp about 270
// instructions (360 would take as long as its bytes at the HBM's rate), so loads and arithmetic
// weigh alike: 32 requests of 4096 positions took 38.9 us, 35.5 without the arithmetic, 34.6
// without the loads.  What a share costs before its first tile (lengths, pages, first tiles, the
// rotated queries: about 4 us) and the joining kernel (2 us) come on top.  Measured with 32 heads
// over 8 of 128: one request of 1025 positions 8.6 us, 32 of up to 4097 26 us (2.8 TB/s); 64 heads,
// 8 of up to 32769 35 us (3.6 TB/s).
//
// The work is the list of (request, head, 64 positions) units in this order; each CTA takes
// an equal, contiguous share of it whatever the lengths are, and a warp of its four one
// 16-position tile of each unit.  A share's segment (its part of one request and head) costs
// about as much beside its tiles as kSegUnits units do, so each (request, head) counts that
// many more, ahead of its first: without them the shares that hold many short requests took
// twice as long as the others (32 requests of 1 to 4096 positions: 38 us, 54% of the SMs' time).
// Measured for 2 / 3 / 5: 29.8 / 28.9 / 27.5 us there, - / 37.7 / 37.2 with 64 heads over 32769.
// A segment that is a whole (request, head) is finished in place; the others leave (max, sum,
// accumulator) partials, which a second kernel adds in the order of the shares.
//   S = K q:     A = K codes (rows positions), B = q (columns the rows)
//   O^T = V^T P: A = V codes (rows channels), B = P transposed in registers
// Tiles come through a ring of kApStages per warp by 16-byte asynchronous copies.
constexpr int kUnit = 16 * kApWarps, kSegUnits = 5;
constexpr int kApStages = 4;
constexpr int kApMaxB = 8192;

// Workspace of the split: prefix sums of the units [B + 1], then two partials per CTA, each
// [8 NT][D + 4] floats (max, sum, 2 unused, accumulator / 2^24).
struct SplitWs {
  int32_t* pref;
  float* part;
};

// Units of request b (0: nothing to do); a request without visible positions still has
// one per head, so that its rows are written.
__device__ __forceinline__ int attn_units(const AttnPagedParams& p, int b, bool flag) {
  int row0, n, kv;
  if (!attn_request(p, b, flag ? p.status : nullptr, row0, n, kv) || n == 0) return 0;
  return p.L.nkv * (kSegUnits + max(1, (kv + kUnit - 1) / kUnit));
}
// First unit of CTA c's share, and the CTA that holds unit u (shares of per or per + 1).
__device__ __forceinline__ int share_begin(int units, int ctas, int c) {
  return c * (units / ctas) + min(c, units % ctas);
}
__device__ __forceinline__ int share_of(int units, int ctas, int u) {
  const int per = units / ctas, rem = units % ctas, cut = rem * (per + 1);
  return u < cut ? u / (per + 1) : rem + (u - cut) / max(per, 1);
}

template <int D, int NT>
struct FewRows {
  static constexpr int kTile = 16 * D + 64;               // K, V and scales of 16 positions
  static constexpr int kRing = kApStages * kTile;         // per warp
  static constexpr int kPW = D + 4;
  static constexpr int kParts = kApWarps * 8 * NT * kPW * 4;  // the warps' partials (over the ring)
  static constexpr int kArea = kApWarps * kRing > kParts ? kApWarps * kRing : kParts;
  static constexpr int kQ = 8 * NT * (D + 8) * 2;          // query operand, rows padded by 16 bytes
  static int smem(int B) { return kArea + kQ + (B + 1) * 4; }
};

template <int D, int NT, bool TREE>
__global__ void __launch_bounds__(kApWarps * 32, NT == 1 ? 4 : 2) attn_few_kernel(const AttnPagedParams p,
                                                                                  const SplitWs ws) {
  using T = FewRows<D, NT>;
  constexpr int KT = D / 16, NPL = D / 32, NJ = D / 32, PW = T::kPW, QS = D + 8;
  extern __shared__ __align__(16) uint8_t few_smem[];
  __shared__ int warp_tot[kApWarps];
  float* part = reinterpret_cast<float*>(few_smem);
  __half* qs = reinterpret_cast<__half*>(few_smem + T::kArea);
  int* pref = reinterpret_cast<int*>(few_smem + T::kArea + T::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  griddep_launch();  // the joining kernel waits for this one's end in any case

  // prefix sums of the requests' units (every CTA for itself)
  {
    const int per = (p.B + kApWarps * 32 - 1) / (kApWarps * 32), b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      pref[b] = sum;  // within the thread's requests, for now
      sum += attn_units(p, b, blockIdx.x == 0);
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += warp_tot[w];
    for (int b = b0; b < b1; ++b) pref[b] += at;
    at += sum;
    if (b1 == p.B && b0 < b1) pref[p.B] = at;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= p.B; b += kApWarps * 32) ws.pref[b] = pref[b];
  }
  const int units = pref[p.B], ctas = gridDim.x;
  int u = share_begin(units, ctas, blockIdx.x);
  const int u_end = share_begin(units, ctas, blockIdx.x + 1);
  if (u == u_end) return;
  int b;
  {
    // the last request whose prefix sum is <= u, by up to three steps of 32 candidates
    b = 0;
    for (int st = p.B > 1024 ? 1024 : p.B > 32 ? 32 : 1; st; st >>= 5) {
      const int i = b + (lane + 1) * st;
      b += st * __popc(__ballot_sync(0xffffffffu, i <= p.B && pref[i] <= u));
    }
  }
  uint8_t* ring = few_smem + warp * T::kRing;

  while (u < u_end) {
    while (pref[b + 1] <= u) ++b;
    const int nv = (pref[b + 1] - pref[b]) / p.L.nkv, nu = nv - kSegUnits, h = (u - pref[b]) / nv;
    const int at = u - pref[b] - h * nv, step = min(nv - at, u_end - u);
    const int k0 = max(at - kSegUnits, 0), k1 = max(at + step - kSegUnits, 0);
    u += step;
    if (k0 == k1) continue;  // the share ends in what the segment costs beside its units
    const int row0 = p.cu[b], n = p.cu[b + 1] - row0, nrow = n * p.G;
    const int kv = attn_length(p, b, nullptr);
    const int* table = p.table + (size_t)b * p.table_stride;
    // the warp's query rows warp, warp + kApWarps, ...: on their way while the pages are looked up
    constexpr int RPW = 8 * NT / kApWarps;
    uint16_t raw[RPW][NPL];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * kApWarps, tok = r / p.G, hh = r - tok * p.G;
      const uint16_t* src = p.q + (row0 + tok) * p.q_stride + (int64_t)(h * p.G + hh) * D;
#pragma unroll
      for (int m = 0; m < NPL; ++m) raw[i][m] = r < nrow ? src[lane + 32 * m] : 0;
    }
    // this warp's tiles: t0, t0 + kApWarps, ... below t1
    const int t0 = k0 * kApWarps + warp, t1 = min(k1 * kApWarps, (kv + 15) / 16);

    // asynchronous copy of one tile into its ring slot; a page outside the pool is left out
    // (its scales are set so that every position is masked).  The page of the tile after it is
    // looked up ahead, so that no copy waits for its address.
    const uint32_t page_bytes = (uint32_t)p.L.nkv * p.L.block, ring0 = smem_u32(ring) + lane * 16;
    const uint8_t* lane_base = p.pages + (size_t)h * p.L.block + lane * 16;
    auto page_at = [&](int t) { return t < t1 ? __ldg(table + ((16 * t) >> p.L.pshift)) : 0; };
    int first_pages[kApStages];
#pragma unroll
    for (int i = 0; i < kApStages; ++i) first_pages[i] = page_at(t0 + i * kApWarps);
    auto load_page = [&](int t, int slot, int page) {
      if (t < t1) {
        const uint32_t pin = (16 * t) & (p.L.psize - 1), d0 = ring0 + slot * T::kTile;
        if ((uint32_t)page < (uint32_t)p.L.npages) {
          const uint8_t* ksrc = lane_base + (uint64_t)(uint32_t)page * page_bytes + pin * (D / 2);
          const uint8_t* vsrc = ksrc + p.L.voff;
#pragma unroll
          for (int i = 0; i < 8 * D; i += 512) {
            cp_async16(d0 + i, ksrc + i);
            cp_async16(d0 + 8 * D + i, vsrc + i);
          }
          if (lane < 4) cp_async16(d0 + 16 * D, ksrc + p.L.soff - pin * (D / 2 - 4));
        } else {
          if (lane == 0) set_status(p.status, FT_DEV_RANGE);
          if (lane < 16) reinterpret_cast<uint32_t*>(ring + slot * T::kTile + 16 * D)[lane] = 0xFFFFFFFFu;  // NaN scales: see below
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kApStages - 1; ++i) load_page(t0 + i * kApWarps, i, first_pages[i]);
    int page_ahead = first_pages[kApStages - 1];
    auto load = [&](int t, int slot) {
      const int page = page_ahead;
      page_ahead = page_at(t + kApWarps);
      load_page(t, slot, page);
    };

    // the rotated query rows as the FP16 operand (channels c % 16 >= 8 divided by 16)
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * kApWarps;
      float v[NPL];
#pragma unroll
      for (int m = 0; m < NPL; ++m) v[m] = bf16_bits_to_f32(raw[i][m]);
      warp_fwht<NPL>(v, p.hb);
      bool bad = false;
#pragma unroll
      for (int m = 0; m < NPL; ++m) {
        const int c = lane + 32 * m;
        const float x = v[m] * p.qscale;
        bad |= !(fabsf(x) <= 65504.0f);
        qs[r * QS + c] = __float2half_rn((c & 8) ? x * 0.0625f : x);
      }
      if (bad) set_status(p.status, FT_DEV_RANGE);
    }
    __syncthreads();
    uint32_t bq[NT][KT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const __half* q0 = qs + (8 * t + g) * QS + 16 * kt + 2 * tig;
        bq[t][kt][0] = *reinterpret_cast<const uint32_t*>(q0);
        bq[t][kt][1] = *reinterpret_cast<const uint32_t*>(q0 + 8);
      }
    // last visible position of this lane's rows (rows past nrow: as the last token's)
    int lim[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) lim[t][i] = kv - n + min((8 * t + 2 * tig + i) / p.G, n - 1);
    const int all = TREE ? kv - n - 1 : kv - n;  // positions up to this are visible to every row

    float acc[NT][KT][4];
    float m[NT][2], l[NT][2], u0[NT][2];  // running max, sum, and max - kPBias (0 for none yet)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      u0[t][0] = u0[t][1] = -kPBias;
      l[t][0] = l[t][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) acc[t][mt][0] = acc[t][mt][1] = acc[t][mt][2] = acc[t][mt][3] = 0.0f;
    }

    int slot = 0;
    for (int t = t0; t < t1; t += kApWarps) {
      cp_async_wait<kApStages - 2>();
      __syncwarp();
      const uint8_t* st = ring + slot * T::kTile;
      const int p0 = 16 * t;
      uint32_t kw[2][NJ], vw[2][NJ];
      const uint8_t* ka = st + g * (D / 2) + tig * (D / 8);
      const uint8_t* va = st + 8 * D + tig * D + (g ^ paged_v_turn<D>(tig)) * (D / 8);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(ka + i * 8 * (D / 2));
          const uint4 c = *reinterpret_cast<const uint4*>(va + i * 4 * D);
          kw[i][0] = a.x, kw[i][1] = a.y, kw[i][2] = a.z, kw[i][3] = a.w;
          vw[i][0] = c.x, vw[i][1] = c.y, vw[i][2] = c.z, vw[i][3] = c.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(ka + i * 8 * (D / 2));
          const uint2 c = *reinterpret_cast<const uint2*>(va + i * 4 * D);
          kw[i][0] = a.x, kw[i][1] = a.y;
          vw[i][0] = c.x, vw[i][1] = c.y;
        }
      }
      const uint32_t sc0 = reinterpret_cast<const uint32_t*>(st + 16 * D)[g];
      const uint32_t sc1 = reinterpret_cast<const uint32_t*>(st + 16 * D)[g + 8];
      // the slot before this one has been read by every lane: refill it
      load(t + (kApStages - 1) * kApWarps, slot == 0 ? kApStages - 1 : slot - 1);
      slot = slot == kApStages - 1 ? 0 : slot + 1;

      float s[NT][4];
#pragma unroll
      for (int c = 0; c < NT; ++c) s[c][0] = s[c][1] = s[c][2] = s[c][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t lo[4], hi[4];
        paged_word(kw[0][j], lo);
        paged_word(kw[1][j], hi);
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          mma_f16(s[c], a0, bq[c][2 * j][0], bq[c][2 * j][1]);
          mma_f16(s[c], a1, bq[c][2 * j + 1][0], bq[c][2 * j + 1][1]);
        }
      }
      const float ks0 = __uint_as_float(sc0 << 16) * kKsUp, ks1 = __uint_as_float(sc1 << 16) * kKsUp;
      const float v0 = __uint_as_float(sc0 & 0xFFFF0000u), v1 = __uint_as_float(sc1 & 0xFFFF0000u);
      const float vs0 = v0 == 0.0f ? kNoScale : fmaxf(v0, kMinScale), vs1 = v1 == 0.0f ? kNoScale : fmaxf(v1, kMinScale);
      // (a scale from 2^110 on, kTooLarge, makes this and with it the scores NaN, whatever they were)
      const float lv0 = fmaf(fmaf(v0, kKsUp, ks0), 0.0f, lg2(vs0)), lv1 = fmaf(fmaf(v1, kKsUp, ks1), 0.0f, lg2(vs1));
      float rs0 = rcp(vs0), rs1 = rcp(vs1);
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        s[c][0] = fmaf(s[c][0], ks0, lv0);
        s[c][1] = fmaf(s[c][1], ks0, lv0);
        s[c][2] = fmaf(s[c][2], ks1, lv1);
        s[c][3] = fmaf(s[c][3], ks1, lv1);
      }
      if (p0 + 15 > all || (sc0 & sc1) == 0xFFFFFFFFu) {  // warp-uniform but for scales of a missing page
        const int pa = p0 + g, pb = pa + 8;
        const bool ga = sc0 != 0xFFFFFFFFu, gb = sc1 != 0xFFFFFFFFu;
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if constexpr (TREE) {
            const int at = p0 - (kv - n);  // the tile's first position among the new tokens
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int tok = min((8 * c + 2 * tig + i) / p.G, n - 1);
              uint32_t bits = tree_bits(p.mask + (row0 + tok) * p.mask_stride, at, n);
              if (at < 0) bits |= at <= -16 ? 0xFFFFu : (1u << -at) - 1u;  // the history
              s[c][i] = ga && ((bits >> g) & 1u) ? s[c][i] : -INFINITY;  // whatever the entry holds
              s[c][2 + i] = gb && ((bits >> (g + 8)) & 1u) ? s[c][2 + i] : -INFINITY;
            }
          } else {
            s[c][0] = ga && pa <= lim[c][0] ? s[c][0] : -INFINITY;  // whatever the entry holds
            s[c][1] = ga && pa <= lim[c][1] ? s[c][1] : -INFINITY;
            s[c][2] = gb && pb <= lim[c][0] ? s[c][2] : -INFINITY;
            s[c][3] = gb && pb <= lim[c][1] ? s[c][3] : -INFINITY;
          }
        }
        // 0 x (1 / scale) of an entry that no row sees must be 0
        if (!ga || pa >= kv) rs0 = 0.0f;
        if (!gb || pb >= kv) rs1 = 0.0f;
      }
      bool move = false;
#pragma unroll
      for (int c = 0; c < NT; ++c)
        move |= fmaxf(s[c][0], s[c][2]) > m[c][0] + kPLazy || fmaxf(s[c][1], s[c][3]) > m[c][1] + kPLazy;
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          float x0 = fmaxf(s[c][0], s[c][2]), x1 = fmaxf(s[c][1], s[c][3]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
          }
          x0 = fmaxf(x0, m[c][0]), x1 = fmaxf(x1, m[c][1]);
          const float f0 = m[c][0] == x0 ? 1.0f : ex2(m[c][0] - x0), f1 = m[c][1] == x1 ? 1.0f : ex2(m[c][1] - x1);
          m[c][0] = x0, m[c][1] = x1;
          u0[c][0] = (x0 == -INFINITY ? 0.0f : x0) - kPBias;
          u0[c][1] = (x1 == -INFINITY ? 0.0f : x1) - kPBias;
          l[c][0] *= f0, l[c][1] *= f1;
#pragma unroll
          for (int mt = 0; mt < KT; ++mt)
            acc[c][mt][0] *= f0, acc[c][mt][1] *= f1, acc[c][mt][2] *= f0, acc[c][mt][3] *= f1;
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const float e0 = ex2(s[c][0] - u0[c][0]), e1 = ex2(s[c][1] - u0[c][1]);
        const float e2 = ex2(s[c][2] - u0[c][0]), e3 = ex2(s[c][3] - u0[c][1]);
        l[c][0] = fmaf(e0, rs0, fmaf(e2, rs1, l[c][0]));
        l[c][1] = fmaf(e1, rs0, fmaf(e3, rs1, l[c][1]));
        const __half2 pa2 = __floats2half2_rn(e0, e1), pb2 = __floats2half2_rn(e2, e3);
        pb[c][0] = movmatrix_trans(v0 == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&pa2));
        pb[c][1] = movmatrix_trans(v1 == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&pb2));
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t lo[4], hi[4];
        paged_word(vw[0][j], lo);
        paged_word(vw[1][j], hi);
        const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]}, a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          mma_f16(acc[c][2 * j], a0, pb[c][0], pb[c][1]);
          mma_f16(acc[c][2 * j + 1], a1, pb[c][0], pb[c][1]);
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // every ring slot is free: the warps' partials go over them
#pragma unroll
    for (int c = 0; c < NT; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[c][0] += __shfl_xor_sync(0xffffffffu, l[c][0], o);
        l[c][1] += __shfl_xor_sync(0xffffffffu, l[c][1], o);
      }
      float* w0 = part + (warp * 8 * NT + 8 * c + 2 * tig) * PW;
      float* w1 = w0 + PW;
      if (g == 0) w0[0] = m[c][0], w0[1] = l[c][0], w1[0] = m[c][1], w1[1] = l[c][1];
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) {
        const int ch = 16 * mt + g;
        w0[4 + ch] = acc[c][mt][0], w1[4 + ch] = acc[c][mt][1];
        w0[4 + ch + 8] = acc[c][mt][2] * 0.0625f, w1[4 + ch + 8] = acc[c][mt][3] * 0.0625f;
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nu;
    // at most one segment of a share continues another share's (slot 0), one other is continued (slot 1)
    float* out = ws.part + (size_t)(2 * blockIdx.x + (k0 == 0 ? 1 : 0)) * (8 * NT * PW);
    for (int r = warp; r < min(8 * NT, nrow); r += kApWarps) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kApWarps; ++w) M = fmaxf(M, part[(w * 8 * NT + r) * PW]);
      float lt = 0.0f, o[NPL] = {};
#pragma unroll
      for (int w = 0; w < kApWarps; ++w) {
        const float* q = part + (w * 8 * NT + r) * PW;
        const float f = q[0] == M ? 1.0f : ex2(q[0] - M);
        lt = fmaf(f, q[1], lt);
#pragma unroll
        for (int i = 0; i < NPL; ++i) o[i] = fmaf(f, q[4 + lane + 32 * i], o[i]);
      }
      if (whole) {
        const float inv = lt == 0.0f ? 0.0f : kOUp / lt;  // a row that sees nothing: zeros
#pragma unroll
        for (int i = 0; i < NPL; ++i) o[i] *= inv;
        warp_fwht<NPL>(o, p.hb);
        const int tok = r / p.G, hh = r - tok * p.G;
        uint16_t* dst = p.o + (row0 + tok) * p.o_stride + (int64_t)(h * p.G + hh) * D;
#pragma unroll
        for (int i = 0; i < NPL; ++i) dst[lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i]));
      } else {
        float* q = out + r * PW;
        if (lane == 0) q[0] = M, q[1] = lt;
#pragma unroll
        for (int i = 0; i < NPL; ++i) q[4 + lane + 32 * i] = o[i];
      }
    }
    __syncthreads();  // part and qs are free again
  }
}

// Joins the partials of the (request, head) pairs that several CTAs shared, W = 1 or 4 warps
// per row, in the order of the shares.
template <int D, int NT, int W>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnPagedParams p, const SplitWs ws, int ctas) {
  constexpr int PW = D + 4, rb = 2 * NT * W;  // CTAs of a pair
  const int r = W == 1 ? 4 * (blockIdx.x % rb) + (threadIdx.x >> 5) : blockIdx.x % rb, bh = blockIdx.x / rb, h = bh % p.L.nkv, b = bh / p.L.nkv;
  const int row0 = p.cu[b], n = p.cu[b + 1] - row0;  // (not the few-rows kernel's: no need to wait)
  griddep_wait();
  const int first = __ldcg(ws.pref + b), next = __ldcg(ws.pref + b + 1), units = __ldcg(ws.pref + p.B);
  if (next == first || r >= n * p.G) return;
  const int nv = (next - first) / p.L.nkv, v0 = first + h * nv;
  const int c0 = share_of(units, ctas, v0 + kSegUnits), c1 = share_of(units, ctas, v0 + nv - 1);
  if (c0 == c1) return;
  const int tok = r / p.G, hh = r - tok * p.G;
  // the first share's partial in its slot 1, the others' in their slot 0
  const float* base = ws.part + (size_t)r * PW;
  join_row<D, W>(p, c1 - c0 + 1, [&](int i) { return base + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * (8 * NT * PW); }, kOUp,
              p.o + (row0 + tok) * p.o_stride + (int64_t)(h * p.G + hh) * D);
}

// CTAs of the few-rows kernel: every SM filled (its occupancy by registers and ring).
static int few_ctas(int nt) {
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  return sms * (nt == 1 ? 4 : 2);
}
// 8-column tiles for max_q tokens of a group of G heads; 0: too many rows for this kernel.
// Trees of more than 16 rows have kernels of their own, ft_attn_tree_few.cu up to 32 and ft_attn_tree.cu above.  Measured,
// this kernel against that of up to 32 rows (us): 32 requests of up to 4096 positions, 32 heads over 8, trees of 4 / 8
// tokens (16 / 32 rows) 36 / 42 and 58 / 45; one of 32768, 64 heads over 8, trees of 2 / 4 tokens 22 / 30 and 33 / 32;
// and that one against the one of more rows, 32 requests of 7 tokens (28 rows) 45 / 61.
static int few_tiles(int max_q, int G) {
  const int64_t rows = (int64_t)max_q * G;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 0;
}

template <int D, int NT, bool TREE>
static cudaError_t launch_few(const AttnPagedParams& p, void* workspace, cudaStream_t st) {
  using T = FewRows<D, NT>;
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_few_kernel<D, NT, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::smem(kApMaxB));
    if (e != cudaSuccess) return e;
    allowed[dev] = 1;
  }
  SplitWs ws;
  ws.pref = static_cast<int32_t*>(workspace);
  ws.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align_up((size_t)(p.B + 1) * 4, 256));
  const int ctas = few_ctas(NT);
  attn_few_kernel<D, NT, TREE><<<ctas, kApWarps * 32, T::smem(p.B), st>>>(p, ws);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // Four warps a row where a pair may have more than twelve partials (a warp loads eight at once).
  // Measured, one against four warps (us; 64 heads over 8): one request of 32768 positions 24.3 / 18.8,
  // of 1024 10.1 / 9.1, four of 32768 37.3 / 35.9, eight 59.9 / 60.5; 32 of 4096 (32 heads) 37.7 / 40.0.
  const bool wide = (int64_t)p.B * p.L.nkv * 12 < ctas;
  cfg.gridDim = dim3((unsigned)(p.B * p.L.nkv * 2 * NT * (wide ? 4 : 1)));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ft_host::pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, wide ? attn_join_kernel<D, NT, 4> : attn_join_kernel<D, NT, 1>, p, ws, ctas);
}

template <bool TREE>
static cudaError_t launch_few_any(const AttnPagedParams& p, int head_dim, int nt, void* ws, cudaStream_t st) {
  if constexpr (!TREE) {
    if (nt == 4) return head_dim == 128 ? launch_few<128, 4, false>(p, ws, st) : launch_few<64, 4, false>(p, ws, st);
  }
  if (head_dim == 128) return nt == 1 ? launch_few<128, 1, TREE>(p, ws, st) : launch_few<128, 2, TREE>(p, ws, st);
  return nt == 1 ? launch_few<64, 1, TREE>(p, ws, st) : launch_few<64, 2, TREE>(p, ws, st);
}

static size_t attn_ws(const ft_block_cfg* c, int B, int total_q, int max_q, bool tree) {
  if (ft_host::check_cfg(c) != FT_OK || B < 1 || B > kApMaxB || total_q < 0 || max_q < 1) return 0;
  const int nt = few_tiles(std::min(max_q, std::max(total_q, 1)), c->n_q / c->n_kv);
  if (tree && (nt == 0 || nt == 4))
    return nt == 0 ? attn_tree_ws(c->n_kv, c->n_q / c->n_kv, c->head_dim, B, total_q) : attn_tree_few_ws(c->n_kv, c->n_q / c->n_kv, c->head_dim, B, total_q);
  if (nt == 0) return attn_tiles_ws(c->n_kv, c->n_q / c->n_kv, c->head_dim, B, total_q);
  return align_up((size_t)(B + 1) * 4, 256) + (size_t)few_ctas(nt) * 2 * (8 * nt) * (c->head_dim + 4) * 4;
}

// Both calls: causal among the new tokens (tree false), or by their masks.
static int attn_call(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const uint16_t* q_bf16, int64_t q_stride,
                     const int32_t* cu_seqlens, const int32_t* kv_len, const int32_t* block_table, int table_stride, bool tree,
                     const uint32_t* mask, int64_t mask_stride, int B, int total_q, int max_q, float scale, uint16_t* o_bf16,
                     int64_t o_stride, void* workspace, size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (B < 1 || total_q < 0 || max_q < 1 || table_stride < 1 || !(scale > 0.0f) || !(scale < 3e38f))
    return FT_ERR_INVALID_ARG;
  if (total_q == 0) return FT_OK;
  const int64_t row = (int64_t)c->n_q * c->head_dim;
  if (!q_bf16 || !o_bf16 || !cu_seqlens || !kv_len || !block_table || !workspace || q_stride < row || o_stride < row)
    return FT_ERR_INVALID_ARG;
  if (!ft_host::aligned16(workspace)) return FT_ERR_INVALID_ARG;
  if (tree && (!mask || (reinterpret_cast<uintptr_t>(mask) & 3u) || mask_stride < ((int64_t)std::min(max_q, total_q) + 31) / 32))
    return FT_ERR_INVALID_ARG;
  if (B > kApMaxB || (int64_t)total_q * (c->n_q / c->n_kv) > INT32_MAX) return FT_ERR_UNSUPPORTED;
  // units of work (a request's and head's positions, one and kSegUnits more) and the joining kernel's CTAs (up
  // to eight a request and head) are counted in 32 bits
  static_assert(1 + kSegUnits <= 8, "units of work");
  if (((int64_t)table_stride * page_size / kUnit + 8) * c->n_kv > INT32_MAX / B) return FT_ERR_UNSUPPORTED;
  if (ws_bytes < attn_ws(c, B, total_q, max_q, tree)) return FT_ERR_WORKSPACE;
  AttnPagedParams p = {};
  p.pages = static_cast<const uint8_t*>(pages);
  p.L = paged_layout(*c, n_pages, page_size);
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
  p.qscale = scale * 1.44269504088896341f * kQUp;
  p.norm = paged_norm(c->had_block);
  p.mask = tree ? mask : nullptr;
  p.mask_stride = mask_stride;
  const int nt = few_tiles(p.max_q, p.G);
  if (tree && (nt == 0 || nt == 4)) {
    if (!attn_tree_fits(p)) return FT_ERR_UNSUPPORTED;
    const cudaError_t e = nt == 0 ? launch_attn_tree(p, c->head_dim, workspace, stream) : launch_attn_tree_few(p, c->head_dim, workspace, stream);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
  }
  if (nt > 0) {
    const cudaError_t e = tree ? launch_few_any<true>(p, c->head_dim, nt, workspace, stream) : launch_few_any<false>(p, c->head_dim, nt, workspace, stream);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
  }
  if (attn_tiles_ctas(p) > INT32_MAX) return FT_ERR_UNSUPPORTED;
  return launch_attn_tiles(p, c->head_dim, workspace, stream) == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // namespace ft

extern "C" {

size_t ft_attn_paged_workspace_bytes(const ft_block_cfg* c, int B, int total_q, int max_q) { return ft::attn_ws(c, B, total_q, max_q, false); }
size_t ft_attn_tree_workspace_bytes(const ft_block_cfg* c, int B, int total_q, int max_q) { return ft::attn_ws(c, B, total_q, max_q, true); }

int ft_attn_paged_int4(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const uint16_t* q_bf16,
                       int64_t q_stride, const int32_t* cu_seqlens, const int32_t* kv_len, const int32_t* block_table,
                       int table_stride, int B, int total_q, int max_q, float scale, uint16_t* o_bf16, int64_t o_stride,
                       void* workspace, size_t ws_bytes, int32_t* dev_status, ft_stream stream) {
  return ft::attn_call(c, pages, n_pages, page_size, q_bf16, q_stride, cu_seqlens, kv_len, block_table, table_stride, false, nullptr, 0, B,
                       total_q, max_q, scale, o_bf16, o_stride, workspace, ws_bytes, dev_status, (cudaStream_t)stream);
}

int ft_attn_tree_paged_int4(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const uint16_t* q_bf16,
                            int64_t q_stride, const int32_t* cu_seqlens, const int32_t* kv_len, const int32_t* block_table,
                            int table_stride, const uint32_t* tree_mask, int64_t mask_stride, int B, int total_q, int max_q,
                            float scale, uint16_t* o_bf16, int64_t o_stride, void* workspace, size_t ws_bytes,
                            int32_t* dev_status, ft_stream stream) {
  return ft::attn_call(c, pages, n_pages, page_size, q_bf16, q_stride, cu_seqlens, kv_len, block_table, table_stride, true, tree_mask,
                       mask_stride, B, total_q, max_q, scale, o_bf16, o_stride, workspace, ws_bytes, dev_status, (cudaStream_t)stream);
}

}  // extern "C"
