// Attention over the paged 4-bit cache for requests with many rows (prompts and chunks
// of prompts), on the fifth-generation tensor cores.
//
// A CTA owns up to 256 rows (tokens x heads of a group, two tiles of M = 128; one tile where
// that leaves SMs without work) of one request and KV head and walks the visible positions,
// or one of several equal parts of them where rows are few, in tiles of 128:
//   S = Q K^T   A = Q from shared memory, B = K codes from shared memory
//   O += P V    A = P from tensor memory (over S's columns), B = V from shared memory
// with FP16 operands and FP32 accumulators in tensor memory (S 2 x 128 columns, O 2 x d
// columns).  K and V are decoded once per CTA for both tiles into the 128-byte-swizzled
// K-major layout; the order of the channels inside a K step is the cache's own, and Q is
// written in the same order.
//
// Scales are multiplied into the operands, relative to a power of two per 32 positions:
// a scale has 8 significant bits and a code 3, so the product is exact in FP16 down to 2^-8
// of that power; where a group has smaller scales its operands are made 2^8 times larger (one
// more product a word, in such groups only) and are exact down to 2^-16.  The groups' powers of
// two, kf for K and 2^f for V, come back as one factor and one term of each score, t = S kf + f:
// P = 2^(t - m) weighs V's operand, and the sum of weights takes 2^-f per group.  (Scales applied per column in the
// softmax needed 96 broadcast 16-byte reads a row and tile, 49 KB of shared-memory bandwidth
// a warp: 5500 cycles per pair of tiles.)
//
// The rotations are products with H too: the query rows go to shared memory as they are (BF16, over
// V's room), Q H comes back from tensor memory as the FP16 operand, and at the end O / l, as two
// BF16 operands, is rotated the same way.  (In registers, by all warps, they took 8.9 and 8.5
// thousand cycles of a CTA of 256 rows, a fifth of its time at 20 tiles; now 5.7 and 4.3.)
//
// Bound by a tile's chain from S over P to the next S: 3600 cycles a pair of tiles, of which the
// tensor core works for 2048 and half of the issue slots are used.  The softmax takes 1500 of the
// chain, so what the issuing warp waits for between P and the next S counts in full: it looks at K and
// V before P is there and commits nothing that another commit says too.  Measured (32 heads over 8 of
// 128): 2 x 2048 tokens over 4096 positions 220 us (935 TFLOP/s), 8192 over 32768 1265 TFLOP/s.
// No faster: P through shared memory, so that the next S need not wait for P V; P V in two halves;
// half tiles with two S by turns (a product with 64 columns takes as long as with 128); two threads a
// row; a second issuing warp; eight decoding warps; decoding left out altogether (3.2 ms, not 3.1, for
// the longer case).
//
// Roles: two warpgroups of softmax (one row per thread, a tile each), one warpgroup
// decoding (the next tile's bytes in flight in registers), one issuing thread.  While one
// tile's softmax runs, the tensor core works for the other:
//   PV0(j) QK0(j+1) PV1(j) QK1(j+1) ...
// The running max moves only when a score passes it by 2^4, so O is rarely rescaled.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
#include <algorithm>

#include "ft_attn_paged.cuh"
#include "ft_tc.cuh"

namespace ft {

namespace tiles {

constexpr int kThreads = 512, kRows = 256, kKeys = 128;
constexpr int kMmaWarp = 12, kPartTiles = 4;
constexpr float kOScale = 512.0f;  // the operands hold V's values x 2^-9
constexpr uint32_t kWide = 0x5C005C00u;  // 2^8 in both halves: the factor of a group with a wide range of scales
constexpr int kScaleRing = 4;  // per tile and group of 32 positions: kf, f, 2^-f, mask of the positions that exist
// Registers of a thread by role (softmax twice, decode, issue): the sum over the four
// warpgroups is what the block is launched with, kThreads x 128.
constexpr int kRegSoftmax = 176, kRegDecode = 96, kRegIssue = 64;
constexpr int kRegCommon = 128;  // before and after the roles
static_assert(2 * kRegSoftmax + kRegDecode + kRegIssue <= 4 * 128, "more registers than the block has");

template <int D>
struct Cfg {
  static constexpr int kQ = 128 * D * 2;                 // one tile's query operand
  static constexpr int kK = kKeys * D * 2, kV = kKeys * D * 2;  // one stage
  static constexpr int kOffQ = 0, kOffK = 2 * kQ, kOffV = kOffK + 2 * kK, kOffH = kOffV + 2 * kV;
  static constexpr int kOffScale = kOffH + D * D * 2;    // H: the rotation's matrix
  static constexpr int kOffBar = kOffScale + kScaleRing * 64;
  static constexpr int kSmem = kOffBar + 256 + 1024;  // 1024: alignment slack
  static constexpr int kColO = 256;                    // tensor memory: S0, S1, then O0, O1
};

}  // namespace tiles

using namespace tiles;

// How the rows and positions are shared out.  With parts > 1 each CTA leaves (max, sum,
// accumulator) partials, [block][head][part][128][D + 4], and meta[block] = (request, first row,
// rows, parts taken: at least kPartTiles tiles each) for the kernel that joins them.
struct TilesSplit {
  int rows, parts;  // rows of a CTA (256; 128 with several parts), parts of the positions
  int4* meta;
  float* part;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnPagedParams p, const TilesSplit sp) {
  using C = Cfg<D>;
  constexpr int NJ = D / 32;
  extern __shared__ uint8_t tiles_smem[];
  const uint32_t raw = smem_u32(tiles_smem);
  uint8_t* sm = tiles_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ int find[5];       // request, first row of the CTA's rows (-1: no work), the request's first row, rows and positions
  __shared__ int warp_tot[16];
  __shared__ uint32_t tmem_slot;
  // (by way of a shuffle the compiler knows that a warp agrees on them: uniform branches and registers)
  auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;

  griddep_launch();  // the joining kernel waits for this one's end in any case
  // ---- which rows: block i of all requests' blocks of rows, the last ones (which see most) first
  const int h = blockIdx.x % p.L.nkv, part = (blockIdx.x / p.L.nkv) % sp.parts, want = blockIdx.x / (p.L.nkv * sp.parts);
  {
    auto blocks = [&](int b, int32_t* status, int& row0, int& n, int& kv) {
      if (!attn_request(p, b, status, row0, n, kv)) return 0;
      return (int)(((int64_t)n * p.G + sp.rows - 1) / sp.rows);
    };
    int32_t* status = blockIdx.x == 0 ? p.status : nullptr;
    if (tid == 0) find[1] = -1;
    __syncthreads();
    // The rotation's matrix as a BF16 operand: row n holds H's entries (+-1, or 0 outside the blocks) of
    // the channel in slot n of the query operand, whose channels have the order of the cache's words.
    auto put_h = [&](int first, int step) {
      for (int i = first; i < D * (D / 8); i += step) {
        const int nn = i / (D / 8), c = i % (D / 8), w = nn / 8, ch = 32 * (w % NJ) + 2 * (w / NJ) + 8 * ((nn % 8) / 2) + (nn & 1);
        const int par = ch & (p.hb - 1);
        uint32_t v[4];
        if (p.hb >= 8) {  // channels 8 c .. 8 c + 7: one block's or another's; the signs of their low three bits
          v[0] = ((ch ^ (8 * c)) < p.hb ? 0x3F803F80u : 0u) ^ ((par & 1) ? 0x80000000u : 0u) ^
                 ((__popc(par & (8 * c)) & 1) ? 0x80008000u : 0u);
          v[1] = v[0] ^ ((par & 2) ? 0x80008000u : 0u);
          v[2] = v[0] ^ ((par & 4) ? 0x80008000u : 0u);
          v[3] = v[1] ^ ((par & 4) ? 0x80008000u : 0u);
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int k = 8 * c + 2 * y;
            const uint32_t a = ((ch ^ k) < p.hb ? 0x3F80u : 0u) | ((uint32_t)__popc(par & k) << 15);
            const uint32_t b = ((ch ^ (k + 1)) < p.hb ? 0x3F80u : 0u) | ((uint32_t)__popc(par & (k + 1)) << 15);
            v[y] = (a & 0xFFFFu) | (b << 16);
          }
        }
        *reinterpret_cast<uint4*>(sm + C::kOffH + chunk_at(D, nn, c)) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    };
    if (p.B <= 32) {  // a request per lane of the first warp
      if (warp > 0) {
        put_h(tid - 32, kThreads - 32);
      } else {
        int row0 = 0, n = 0, kv = 0;
        const int nb = lane < p.B ? blocks(lane, status, row0, n, kv) : 0;
        int inc = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        const int i = __shfl_sync(0xffffffffu, inc, 31) - 1 - want;
        if (i >= inc - nb && i < inc) {
          find[0] = lane, find[2] = row0, find[3] = n, find[4] = kv;
          find[1] = (i - (inc - nb)) * sp.rows;
        }
      }
    } else {
      put_h(tid, kThreads);
      const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
      int sum = 0, row0, n, kv;
      for (int b = b0; b < b1; ++b) sum += blocks(b, status, row0, n, kv);
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) warp_tot[warp] = inc;
      __syncthreads();
      int at = inc - sum, total = 0;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += warp_tot[w];
        total += warp_tot[w];
      }
      const int i = total - 1 - want;
      if (i >= at && i < at + sum) {
        for (int b = b0; b < b1; ++b) {
          const int nb = blocks(b, nullptr, row0, n, kv);
          if (i < at + nb) {
            find[0] = b, find[2] = row0, find[3] = n, find[4] = kv;
            find[1] = (i - at) * sp.rows;
            break;
          }
          at += nb;
        }
      }
    }
    __syncthreads();
  }
  const int b = uni(find[0]), r0 = uni(find[1]), row0 = uni(find[2]), n = uni(find[3]), kv = uni(find[4]);
  if (r0 < 0) {
    if (sp.parts > 1 && h == 0 && part == 0 && tid == 0) sp.meta[want] = make_int4(0, 0, 0, 0);
    return;
  }
  const int nrow = (int)min((int64_t)n * p.G - r0, (int64_t)sp.rows);  // rows of this CTA
  const int ntile = nrow > 128 ? 2 : 1;
  const int last = kv - n + (r0 + nrow - 1) / p.G;               // last visible position of any row
  const int all_kt = last >= 0 ? last / kKeys + 1 : 0;
  const int parts = min(sp.parts, max(1, (all_kt + kPartTiles - 1) / kPartTiles)), per_part = parts == 1 ? all_kt : (all_kt + parts - 1) / parts;
  const int j0 = part * per_part, nkt = max(0, min(all_kt - j0, per_part));  // this CTA's tiles: j0, j0 + 1, ...
  if (sp.parts > 1 && h == 0 && part == 0 && tid == 0) sp.meta[want] = make_int4(b, r0, nrow, parts);
  if (part >= parts) return;
  const int* table = p.table + (size_t)b * p.table_stride;

  // ---- the query rows as they are (BF16), zeros behind the last, to V's room: the tensor core rotates them
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  // each thread's chunks: one of every kStep-th row, its token and head of the group advanced along
  constexpr int kStep = kThreads / kChunks;
  auto walk = [&](int rows, auto&& body) {  // body(row, chunk, token's row of q and o, first element in it)
    const int c = tid % kChunks, rg = r0 + tid / kChunks, dt = kStep / p.G, dh = kStep - dt * p.G;
    int tok = rg / p.G, hh = rg - tok * p.G;
#pragma unroll 4
    for (int rr = tid / kChunks; rr < rows; rr += kStep) {
      body(rr, c, row0 + tok, (h * p.G + hh) * D + 8 * c);
      tok += dt, hh += dh;
      if (hh >= p.G) hh -= p.G, ++tok;
    }
  };
  if (nkt > 0) {
    walk(128 * ntile, [&](int rr, int c, int token, int at) {
      const uint16_t* src = p.q + (rr < nrow ? token * p.q_stride + at : 0);
      const uint32_t to = C::kOffV + (rr >= 128 ? C::kQ : 0) + chunk_at(128, rr & 127, c);
      if (rr >= nrow || (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        cp_async16_zfill(sm32 + to, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15), rr < nrow);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = (uint32_t)src[2 * k] | ((uint32_t)src[2 * k + 1] << 16);
        *reinterpret_cast<uint4*>(sm + to) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    });
  }
  const uint32_t bar = sm32 + C::kOffBar;
  const uint32_t s_full = bar, p_full = bar + 16, o_full = bar + 32, k_full = bar + 48, k_empty = bar + 64,
                 v_full = bar + 80, sc_full = bar + 96, drained = bar + 128, rot_full = bar + 136, rows_put = bar + 152;
  // (rot_full, rows_put: twice each, the queries' rotation and the outputs')
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(k_full + 8 * i, 128);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 128);
      mbar_init(rot_full + 8 * i, 1);
      mbar_init(rows_put + 8 * i, 128);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full + 8 * i, 128);
    mbar_init(drained, 1);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  cp_async_wait_all();
  fence_proxy_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  auto out_at = [&](int r, int c) { return (uint32_t)((r * kChunks + (c ^ (r & 7))) << 4); };  // chunk c of row r on its way out
  float4* scales = reinterpret_cast<float4*>(sm + C::kOffScale);  // [ring][kf, f, 2^-f, mask][4 groups]
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax: one row per thread
    regs_up<kRegSoftmax>();
    const int t = warp >> 2, row = tid & 127, r = r0 + 128 * t + row;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    if (t < ntile) {
      const int tok = min(r / p.G, n - 1);
      const int lim = kv - n + tok;  // last position this row sees
      const int lim_all = kv - n + (r0 + 128 * t + 32 * (warp & 3)) / p.G;  // and that every row of the warp sees
      // the rotated query row as the FP16 operand
      if (nkt > 0 && !all_wait(rot_full + 8 * t, 0)) ok = false;
      if (ok && nkt > 0) {
        fence_after();
        const float f0 = p.qscale * p.norm;
        uint32_t over = 0u;  // stays zero unless a value is infinite or NaN in FP16
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_base + 128 * t + c, v);
          wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 hv = __floats2half2_rn(__uint_as_float(v[8 * i + 2 * k]) * f0, __uint_as_float(v[8 * i + 2 * k + 1]) * f0);
              o[k] = *reinterpret_cast<const uint32_t*>(&hv);
              over = hfma2(o[k], 0u, over);
            }
            *reinterpret_cast<uint4*>(sm + C::kOffQ + C::kQ * t + chunk_at(128, row, c / 8 + i)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        if ((over & 0x7FFF7FFFu) != 0u) set_status(p.status, FT_DEV_RANGE);
        fence_proxy_async_smem();
        fence_before();
        mbar_arrive(rows_put + 8 * t);
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; ok && j < nkt; ++j) {
        if (!all_wait(s_full + 8 * t, j & 1) || !all_wait(sc_full + 8 * (j % kScaleRing), (j / kScaleRing) & 1)) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(tmem + lane_base + 128 * t + c, s + c);
        const float4* sc = scales + 4 * (j % kScaleRing);
        const float4 kf4 = sc[0], f4 = sc[1], rf4 = sc[2];
        const uint4 mask4 = reinterpret_cast<const uint4*>(sc)[3];
        const float kf[4] = {kf4.x, kf4.y, kf4.z, kf4.w}, f[4] = {f4.x, f4.y, f4.z, f4.w}, rf[4] = {rf4.x, rf4.y, rf4.z, rf4.w};
        wait_ld();
        // a tile that some row of the warp sees in part, or with positions on a page outside the pool
        if (kKeys * (j0 + j) + kKeys - 1 > lim_all || (mask4.x & mask4.y & mask4.z & mask4.w) != 0xFFFFFFFFu) {
          const uint32_t mask[4] = {mask4.x, mask4.y, mask4.z, mask4.w};
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            s[c] = kKeys * (j0 + j) + c <= lim && ((mask[c / 32] >> (c % 32)) & 1u) ? s[c] : 0xFF800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float q[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 32 * g; c < 32 * g + 32; c += 4)
#pragma unroll
            for (int k = 0; k < 2; ++k) q[k] = max3(q[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
          mx = fmaxf(mx, fmaf(fmaxf(q[0], q[1]), kf[g], f[g]));
        }
        const bool need = mx > m + kPLazy;
        if (__any_sync(0xffffffffu, need)) {
          const float to = need ? mx : m;
          const float fac = to == m ? 1.0f : ex2(m - to);
          m = to;
          if (j > 0) {
            l *= fac;  // (S came after the last product into O, which is done)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
              tmem_st32(tmem + lane_base + C::kColO + D * t + c, o);
            }
          }
        }
        const float u = kPBias - (m == -INFINITY ? 0.0f : m);
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          uint32_t o[32];
#pragma unroll
          for (int g = 2 * g2; g < 2 * g2 + 2; ++g) {
            const f32x2 kf2(kf[g], kf[g]), u2(u + f[g], u + f[g]);
            f32x2 sum[2] = {f32x2(0.0f, 0.0f), f32x2(0.0f, 0.0f)};
#pragma unroll
            for (int c = 32 * g; c < 32 * g + 32; c += 2) {
              float x0, x1;
              fma2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), kf2, u2).get(x0, x1);
              x0 = ex2(x0), x1 = ex2(x1);
              sum[(c / 2) & 1] = add2(sum[(c / 2) & 1], f32x2(x0, x1));
              const __half2 hv = __floats2half2_rn(x0, x1);
              o[(c - 64 * g2) / 2] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            float a, c;
            add2(sum[0], sum[1]).get(a, c);
            l = fmaf(a + c, rf[g], l);
          }
          tmem_st32(tmem + lane_base + 128 * t + 32 * g2, o);
        }
        wait_st();
        fence_before();
        mbar_arrive(p_full + 8 * t);
      }
      if (ok && nkt > 0 && !all_wait(o_full + 8 * t, 0)) ok = false;
      if (ok && parts > 1) {
        // ---- this part's maximum, sum and O for the joining kernel
        fence_after();
        float* partial = sp.part + ((((size_t)want * p.L.nkv + h) * sp.parts + part) * 128 + row) * (D + 4);
        partial[0] = m, partial[1] = l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (nkt > 0) {
            tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
            wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(partial + 4 + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      } else if (ok && nkt > 0) {
        // ---- O / l as two BF16 operands, the value and what its rounding left (2^-17 remains), over those
        // of QK, which are done with (tile 0 takes Q's room, tile 1 K's); rotated by the tensor core
        fence_after();
        const float inv = l == 0.0f ? 0.0f : kOScale / l;  // a row that sees nothing: zeros
        uint8_t* own = sm + (t == 0 ? C::kOffQ : C::kOffK);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
          wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = __uint_as_float(o[8 * i + 2 * k]) * inv, b = __uint_as_float(o[8 * i + 2 * k + 1]) * inv;
              const __nv_bfloat162 hv = __floats2bfloat162_rn(a, b);
              hi[k] = *reinterpret_cast<const uint32_t*>(&hv);
              const __nv_bfloat162 lv = __floats2bfloat162_rn(a - __uint_as_float(hi[k] << 16), b - __uint_as_float(hi[k] & 0xFFFF0000u));
              lo[k] = *reinterpret_cast<const uint32_t*>(&lv);
            }
            const uint32_t at = chunk_at(128, row, c / 8 + i);
            *reinterpret_cast<uint4*>(own + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(own + C::kQ + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        fence_before();
        mbar_arrive(rows_put + 8 * t);
        if (!all_wait(rot_full + 8 * t, 1)) ok = false;
        if (ok) {
          fence_after();
          // slots back to channels: chunk e of group jj holds its pairs of four words
#pragma unroll
          for (int jj = 0; jj < NJ; ++jj) {
            uint32_t v[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld8(tmem + lane_base + 128 * t + 8 * (q * NJ + jj), v[q]);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 bv = __floats2bfloat162_rn(__uint_as_float(v[q][2 * e]) * p.norm, __uint_as_float(v[q][2 * e + 1]) * p.norm);
                w[q] = *reinterpret_cast<const uint32_t*>(&bv);
              }
              *reinterpret_cast<uint4*>(own + out_at(row, 4 * jj + e)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
    regs_down<kRegCommon>();
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ decode K and V
    regs_down<kRegDecode>();
    const int w4 = warp - 8;  // positions 32 w4 .. 32 w4 + 31 of each tile
    constexpr int NW = D == 128 ? 4 : 2;  // words of a K piece; V words a lane takes of a group of 8 positions
    // Group i (positions 8 i .. 8 i + 7 of the warp's): this lane's K piece is (position lane & 7, column
    // lane >> 3); its V words are those of channels (g = lane & 7, j = lane >> 3) for the four pairs,
    // for d = 64 (j = (lane >> 3) & 1) for two of them.  Scales and pages belong to position `lane`.
    uint32_t kw[4][NW], vw[4][NW], sc = 0u;
    int page = -1, page_next = -1;
    bool there = false;
    const uint32_t page_bytes = (uint32_t)p.L.nkv * p.L.block;
    const uint8_t* base = p.pages + (size_t)h * p.L.block;
    const int k_lane = (lane & 7) * (D / 2) + (lane >> 3) * (D / 8);
    int v_lane[NW];  // of pair k (d = 64: of the lane half's two); the chunks' turn repeats every four pairs
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int pair = D == 128 ? k : 2 * (lane >> 4) + k, jj = D == 128 ? lane >> 3 : (lane >> 3) & 1;
      v_lane[k] = pair * D + ((lane & 7) ^ paged_v_turn<D>(pair)) * (D / 8) + 4 * jj;
    }
    auto page_of = [&](int j) {  // raw entry; positions behind the end: -1
      const int pos = kKeys * (j0 + j) + 32 * w4 + lane;
      return pos < kv ? __ldg(table + (pos >> p.L.pshift)) : -1;
    };
    // bytes of tile j on their way into registers; the pages of tile j + 1 are looked up with them
    auto load_k = [&](int j) {
      page = page_next;
      const int pos = kKeys * (j0 + j) + 32 * w4 + lane;
      there = pos < kv && (uint32_t)page < (uint32_t)p.L.npages;
      if (pos < kv && !there) set_status(p.status, FT_DEV_RANGE);
      if (!there) page = -1;
      sc = there ? ld_stream_u32(base + (uint64_t)(uint32_t)page * page_bytes + p.L.soff + 4 * (pos & (p.L.psize - 1))) : 0u;
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // 16 positions, on one page
        const int pg = __shfl_sync(0xffffffffu, page, 16 * q), pin = (kKeys * (j0 + j) + 32 * w4 + 16 * q) & (p.L.psize - 1);
        const uint8_t* src = base + (uint64_t)(uint32_t)pg * page_bytes + pin * (D / 2) + k_lane;
#pragma unroll
        for (int i = 2 * q; i < 2 * q + 2; ++i) {
#pragma unroll
          for (int k = 0; k < NW; ++k) kw[i][k] = 0u;
          if (pg >= 0) {
            if constexpr (D == 128) {
              const uint4 x = ld_stream_v4(src + (i & 1) * 8 * (D / 2));
              kw[i][0] = x.x, kw[i][1] = x.y, kw[i][2] = x.z, kw[i][3] = x.w;
            } else {
              const uint2 x = ld_stream_v2(src + (i & 1) * 8 * (D / 2));
              kw[i][0] = x.x, kw[i][1] = x.y;
            }
          }
        }
      }
    };
    auto load_v = [&](int j) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int pg = __shfl_sync(0xffffffffu, page, 16 * q), pin = (kKeys * (j0 + j) + 32 * w4 + 16 * q) & (p.L.psize - 1);
        const uint8_t* src = base + (uint64_t)(uint32_t)pg * page_bytes + p.L.voff + pin * (D / 2);
#pragma unroll
        for (int i = 2 * q; i < 2 * q + 2; ++i)
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            vw[i][k] = 0u;
            if (pg >= 0) vw[i][k] = ld_stream_u32(src + (i & 1) * 4 * D + v_lane[k]);
          }
      }
      page_next = page_of(j + 1);
    };
    if (nkt > 0) {
      page_next = page_of(0);
      load_k(0);
      load_v(0);
    }
    for (int j = 0; j < nkt; ++j) {
      const int st = j & 1;
      // An entry with a scale from 2^110 on, or one that is not finite (nor was its own row), makes the rows that see
      // it NaN, but must not reach its neighbours, nor the rows that do not see it: its K operand is NaN, which is
      // one column of S, masked like any other, and its V operand is 0.
      const bool poor = (sc & 0x7FFFu) >= kTooLarge || ((sc >> 16) & 0x7FFFu) >= kTooLarge;
      if (poor) sc = 0u;
      // the 32 positions' scales relative to their largest's power of two, as multipliers of the
      // decoded words (codes x 2^-24 and, for odd values, x 2^-20): code x (scale / 2^e) x 2^-9,
      // or x 2^-1 where a scale's exponent is more than 7 below the largest's
      const uint32_t xk = (sc & 0x7FFFu) >> 7, xv = (sc >> 23) & 0xFFu;
      uint32_t ek = __reduce_max_sync(0xffffffffu, xk), ev = __reduce_max_sync(0xffffffffu, xv);
      const bool wide_k = __any_sync(0xffffffffu, xk != 0u && xk + 7u < ek);
      const bool wide_v = __any_sync(0xffffffffu, xv != 0u && xv + 7u < ev);
      ek = max(ek, 27u), ev = ev == 0u ? kNoScaleExp : max(ev, 27u);
      const float mk = poor ? __uint_as_float(0x7FC00000u) : __uint_as_float(sc << 16) * __uint_as_float((268u - ek) << 23);
      const float mv = __uint_as_float(sc & 0xFFFF0000u) * __uint_as_float((268u - ev) << 23);
      const __half2 mk2 = __floats2half2_rn(mk, mk * 0.0625f);  // (even, odd values)
      const uint32_t mku = *reinterpret_cast<const uint32_t*>(&mk2);
      const float mv_next = __shfl_down_sync(0xffffffffu, mv, 1);
      const __half2 mv2 = __floats2half2_rn(mv, mv_next);  // at even lanes: a pair of positions
      const uint32_t mvu = *reinterpret_cast<const uint32_t*>(&mv2);
      const uint32_t exist = __ballot_sync(0xffffffffu, there);
      if (j >= 2 && !all_wait(k_empty + 8 * st, ((j - 2) >> 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        float* dst = reinterpret_cast<float*>(scales + 4 * (j % kScaleRing)) + w4;
        const uint32_t tv = wide_v ? ev - 8u : ev;
        dst[0] = __uint_as_float((wide_k ? ek - 4u : ek + 4u) << 23);  // 2^(e + 9) / kQUp (or 2^-8 of it), e = ek - 126
        dst[4] = (float)((int)tv - 126);
        dst[8] = __uint_as_float((253u - tv) << 23);
        dst[12] = __uint_as_float(exist);
      }
      {
        uint8_t* kd = sm + C::kOffK + st * C::kK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * w4 + 8 * i + (lane & 7);
          const uint32_t both = __shfl_sync(0xffffffffu, mku, 8 * i + (lane & 7));
          const uint32_t m0 = prmt(both, both, 0x1010u), m1 = prmt(both, both, 0x3232u);
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const int w = (lane >> 3) * NJ + k;  // word of the entry: slots 8 w .. 8 w + 7 of the operand's row
            uint32_t r[4];
            paged_word(kw[i][k], r);
            if (wide_k) {
#pragma unroll
              for (int e = 0; e < 4; ++e) r[e] = hmul2(r[e], kWide);
            }
            *reinterpret_cast<uint4*>(kd + (w / 8) * (kKeys * 128) + key * 128 + (((w % 8) ^ (key & 7)) << 4)) =
                make_uint4(hmul2(r[0], m0), hmul2(r[1], m1), hmul2(r[2], m0), hmul2(r[3], m1));
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(sc_full + 8 * (j % kScaleRing));
      mbar_arrive(k_full + 8 * st);
      if (j + 1 < nkt) load_k(j + 1);
      // (QK of tile j - 1 was issued behind PV of tile j - 2; before that V's room held the query rows)
      if (j >= 2 ? !all_wait(k_empty + 8 * (st ^ 1), ((j - 1) >> 1) & 1) : st < ntile && !all_wait(rot_full + 8 * st, 0)) {
        ok = false;
        break;
      }
      {
        uint8_t* vd = sm + C::kOffV + st * C::kV;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int chunk = 4 * w4 + i;  // 8 positions
          uint8_t* panel = vd + (chunk / 8) * (D * 128);
          uint32_t r[NW][4];
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const uint32_t m0 = __shfl_sync(0xffffffffu, mvu, 8 * i + 2 * (D == 128 ? k : 2 * (lane >> 4) + k));
            const uint32_t m1 = hmul2(m0, 0x2C002C00u);  // / 16
            paged_word(vw[i][k], r[k]);
            if (wide_v) {
#pragma unroll
              for (int e = 0; e < 4; ++e) r[k][e] = hmul2(r[k][e], kWide);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) r[k][e] = hmul2(r[k][e], (e & 1) ? m1 : m0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = 32 * (D == 128 ? lane >> 3 : (lane >> 3) & 1) + (lane & 7) + 8 * e;
            uint8_t* dst = panel + ch * 128 + (((chunk % 8) ^ (ch & 7)) << 4);
            if constexpr (D == 128)
              *reinterpret_cast<uint4*>(dst) = make_uint4(r[0][e], r[1][e], r[2][e], r[3][e]);
            else
              *reinterpret_cast<uint2*>(dst + 8 * (lane >> 4)) = make_uint2(r[0][e], r[1][e]);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(v_full + 8 * st);
      if (j + 1 < nkt) load_v(j + 1);
    }
  } else {
    regs_down<kRegIssue>();
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------- tensor-core issue
      constexpr uint32_t id_qk = idesc_f16(128, kKeys), id_pv = idesc_f16(128, D), id_rot = idesc_bf16(128, D);
      const uint32_t lead = lane == 0 ? 1u : 0u, tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = desc_lo(sm32 + C::kOffQ), k_lo = desc_lo(sm32 + C::kOffK), v_lo = desc_lo(sm32 + C::kOffV);
      auto qk = [&](int t, int j) {
        const uint32_t qa = q_lo + t * (C::kQ >> 4), ka = k_lo + (j & 1) * (C::kK >> 4), d = tm + 128 * t;
        mma_ss<false>(d, qa, ka, id_qk, lead);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks) {
          const uint32_t o = ((ks / 4) * (128 * 128) + 32 * (ks % 4)) >> 4;
          mma_ss<true>(d, qa + o, ka + o, id_qk, lead);
        }
        commit(s_full + 8 * t, lead);
      };
      auto pv = [&](int t, int j) {
        const uint32_t va = v_lo + (j & 1) * (C::kV >> 4), d = tm + C::kColO + D * t, pa = tm + 128 * t;
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_ts(d, pa + 8 * ks, va + (((ks / 4) * (D * 128) + 32 * (ks % 4)) >> 4), id_pv, ks > 0 ? 1u : (uint32_t)j, lead);
      };
      // rows times H, over S's columns; the rows' n operands one after another
      auto rotate = [&](int t, uint32_t rows_at, int n) {
        const uint32_t h_lo = desc_lo(sm32 + C::kOffH), d = tm + 128 * t;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t ra = desc_lo(sm32 + rows_at + i * C::kQ);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t a = ra + (((ks / 4) * (128 * 128) + 32 * (ks % 4)) >> 4), b = h_lo + (((ks / 4) * (D * 128) + 32 * (ks % 4)) >> 4);
            if (ks == 0 && i == 0) mma_ss<false>(d, a, b, id_rot, lead);
            else mma_ss<true>(d, a, b, id_rot, lead);
          }
        }
        commit(rot_full + 8 * t, lead);
      };
      if (nkt > 0) {
        for (int t = 0; t < ntile; ++t) rotate(t, C::kOffV + t * C::kQ, 1);
        ok = all_wait(k_full, 0);
        for (int t = 0; ok && t < ntile; ++t) {
          ok = all_wait(rows_put + 8 * t, 0);
          if (!ok) break;
          fence_after();
          qk(t, 0);
        }
        if (ok) commit(k_empty, lead);
      }
      // What can be waited for before P is there is waited for then, and few things are committed: S of tile j
      // says that PV of tile j - 1 is done too, as does k_empty for V's room.
      for (int j = 0; ok && j < nkt; ++j) {
        const bool more = j + 1 < nkt;
        ok = all_wait(v_full + 8 * (j & 1), (j >> 1) & 1) && (!more || all_wait(k_full + 8 * ((j + 1) & 1), ((j + 1) >> 1) & 1));
        for (int t = 0; ok && t < ntile; ++t) {
          ok = all_wait(p_full + 8 * t, j & 1);
          if (!ok) break;
          fence_after();
          pv(t, j);
          if (more) qk(t, j + 1);
          else commit(o_full + 8 * t, lead);
        }
        if (ok && more) commit(k_empty + 8 * ((j + 1) & 1), lead);
      }
      for (int t = 0; ok && nkt > 0 && parts == 1 && t < ntile; ++t) {
        ok = all_wait(rows_put + 8 * t, 1);
        if (!ok) break;
        fence_after();
        rotate(t, t == 0 ? C::kOffQ : C::kOffK, 2);
      }
      // tensor memory is freed only when nothing issued here is in flight
      commit(drained, lead);
      if (!all_wait(drained, 0)) ok = false;
    }
  }
  if (!ok) set_status(p.status, FT_DEV_TIMEOUT);
  fence_before();
  const bool all_ok = __syncthreads_and(ok);
  fence_after();
  // Only now may the others take registers again: the softmax warps have given theirs back before
  // the barrier.  (Taken earlier, by warps that are through before a softmax warp has come to
  // take its share, they would leave that warp waiting for registers that nobody returns.)
  if (warp >= 8) regs_up<kRegCommon>();
  // ---- the rows stored, by all warps
  if (all_ok && parts == 1) {
    walk(nrow, [&](int rr, int c, int token, int at) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);  // nothing visible: zeros
      if (nkt > 0) v = *reinterpret_cast<const uint4*>(sm + (rr < 128 ? C::kOffQ : C::kOffK) + out_at(rr & 127, c));
      uint16_t* dst = p.o + token * p.o_stride + at;
      if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[2 * k] = (uint16_t)w[k], dst[2 * k + 1] = (uint16_t)(w[k] >> 16);
      }
    });
  }
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

// Joins the parts of each row, a warp per row.
template <int D>
__global__ void __launch_bounds__(128) attn_tiles_join_kernel(const AttnPagedParams p, const TilesSplit sp) {
  griddep_wait();
  const int h = blockIdx.y, r = 4 * (blockIdx.x % 32) + (threadIdx.x >> 5), block = blockIdx.x / 32;
  const int4 meta = __ldcg(sp.meta + block);
  if (r >= meta.z || meta.w == 1) return;
  const int rg = meta.y + r, tok = rg / p.G, hh = rg - tok * p.G;
  const float* base = sp.part + (((size_t)block * p.L.nkv + h) * sp.parts * 128 + r) * (D + 4);
  join_row<D>(p, meta.w, [&](int i) { return base + (size_t)i * 128 * (D + 4); }, kOScale,
              p.o + (p.cu[meta.x] + tok) * p.o_stride + (int64_t)(h * p.G + hh) * D);
}

// Rows of a CTA and parts of the positions, from what the host knows (an upper bound of the
// blocks of all requests).  128 rows where all blocks then still run at once, and as many
// parts as fill the SMs (up to 16, counting half a block for the requests' remainders).  Measured,
// 256 rows and one part against this rule (us): 256 tokens over 32768 positions (8B shape) 505 / 229,
// 64 of each of four requests over 8192 139 / 73, 2000 over 3000 with 4 heads 63 / 38; 5 requests of
// 777 (8 heads, d 64) run at once only with 256 rows, 21.5 (128 rows: 32.6).  Not built: 256 rows with
// parts.  A 128-row CTA's tile takes nearly as long as one of 256 rows (3400 and 3600 cycles), so 256 to 768
// tokens over a long history leave time: 226, 428 (512), 477 (640: one part again) and 481 us over 32768.
static void tiles_shape(int nkv, int G, int B, int total_q, int& rows, int& parts, int64_t& blocks) {
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  const int64_t all = (int64_t)total_q * G, some = std::min(B, total_q);
  rows = kRows, parts = 1;
  blocks = all / kRows + some;
  if ((all / 128 + some) * nkv > sms) return;
  rows = 128;
  blocks = all / 128 + some;
  const int64_t likely = std::max<int64_t>(1, (2 * (all / 128) + some) * nkv / 2);
  parts = (int)std::min<int64_t>(16, std::max<int64_t>(1, (sms + likely / 2) / likely));
}

size_t attn_tiles_ws(int nkv, int G, int head_dim, int B, int total_q) {
  int rows, parts;
  int64_t blocks;
  tiles_shape(nkv, G, B, std::max(total_q, 1), rows, parts, blocks);
  if (parts == 1) return 16;
  return align_up((size_t)blocks * 16, 256) + (size_t)blocks * nkv * parts * 128 * (head_dim + 4) * 4;
}

int64_t attn_tiles_ctas(const AttnPagedParams& p) {
  int rows, parts;
  int64_t blocks;
  tiles_shape(p.L.nkv, p.G, p.B, p.total_q, rows, parts, blocks);
  return blocks * p.L.nkv * parts;
}

template <int D>
static cudaError_t launch_tiles_d(const AttnPagedParams& p, void* workspace, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    // the roles' register shares add up to 128 a thread: a build with fewer would wait for them forever
    cudaFuncAttributes fa = {};
    if (cudaFuncGetAttributes(&fa, attn_tiles_kernel<D>) != cudaSuccess) return cudaErrorInvalidDeviceFunction;
    if (fa.numRegs < kRegCommon) return cudaErrorInvalidConfiguration;
    allowed[dev] = 1;
  }
  TilesSplit sp = {};
  int64_t blocks;
  tiles_shape(p.L.nkv, p.G, p.B, p.total_q, sp.rows, sp.parts, blocks);
  sp.meta = static_cast<int4*>(workspace);
  sp.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align_up((size_t)blocks * 16, 256));
  attn_tiles_kernel<D><<<(unsigned)(blocks * p.L.nkv * sp.parts), kThreads, Cfg<D>::kSmem, st>>>(p, sp);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || sp.parts == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks * 32, p.L.nkv);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ft_host::pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_tiles_join_kernel<D>, p, sp);
}

cudaError_t launch_attn_tiles(const AttnPagedParams& p, int head_dim, void* workspace, cudaStream_t st) {
  return head_dim == 128 ? launch_tiles_d<128>(p, workspace, st) : launch_tiles_d<64>(p, workspace, st);
}

}  // namespace ft
