// Attention of drafted token trees over the paged 4-bit cache, on the fifth-generation tensor cores.
//
// The formulas are at the top of ft_attn_paged.cuh; which of the new tokens a token sees is in its mask's bits.
//
// How the work is shared out over the CTAs, one an SM, and joined: ft_attn_tree.cuh.
//
// Inside a CTA two tiles of products run against each other, the tensor core working for one while the other's
// softmax runs: where a block has more than 128 rows, its two halves over the same positions, else the same rows
// over positions by turns (tile 0 the even ones, tile 1 the odd), added up at the segment's end.
//   S = Q K^T   A = Q from shared memory, B = K codes from shared memory
//   O += P V    A = P from tensor memory (over S's columns), B = V from shared memory
// Operands, their scales and the softmax are those of ft_attn_tiles.cu.
//
// Three launches, each behind its predecessor's start: the requests' prefix sums and the query rows, rotated and rounded
// to FP16; this kernel; the joining one.
//
// Roles: two warpgroups of softmax (one row per thread, a tile each), two decoding K and V (a tile's bytes in flight in
// registers while the one before it is decoded), a warp that works out the segments ahead, one that copies the query
// rows, and two that issue the products.
//
// Bound by the chain from S over P to the next S: 4400 cycles a pair of tiles, of which the tensor core works for 2048,
// while decoding keeps up (2 x 1250).  Leaving out the weights' 2^x, the decoding's stores or most of the products makes
// 5 to 8% each.  Where products and decoding meet at shared memory (a product of two operands in it takes all of its 128
// bytes a cycle) both wait.  Measured: one tree of 64 tokens over 32768 positions, 64 heads over 8 of 128, 85 us of the
// three kernels (804 TFLOP/s; with the kernel for prompts and chunks, masked, 124); a segment takes about as long as eight units beside its
// positions (4: 80 us where 8 takes 70, 32 requests of up to 4096; 12 and 18: 70 and 74).
// Slower: all of S kept in registers by the softmax (a warpgroup less for decoding, 136 us), code unrolled (see below),
// P handed over as a whole (93 us) or from its first half on (135: the turn is then held while the rest is made).
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
#include <algorithm>
#include <type_traits>

#include "ft_attn_tree.cuh"

namespace ft {

namespace tree {

constexpr int kThreads = 640;
constexpr int kAheadWarp = 16, kMmaWarp = 18;  // (the first schedulers have the softmax's warps of few rows)
constexpr int kSegUnits = 8;  // a segment's cost beside its positions, in units of 128 rows x 128 positions
constexpr int kWorks = 4;     // segments known ahead: decoding looks up to two beyond its own, never behind the query rows'
constexpr float kOScale = 512.0f;  // the operands hold V's values x 2^-9
constexpr uint32_t kWide = 0x5C005C00u;  // 2^8 in both halves: the factor of a group with a wide range of scales
constexpr int kScaleRing = 4;  // per tile and group of 32 positions: kf, f, 2^-f, mask of the positions that exist
// Registers of a thread by role (softmax twice, decode twice, the others): the sum over the five warpgroups is what the
// block is launched with, kThreads x kRegLaunch.
constexpr int kRegSoftmax = 112, kRegDecode = 80, kRegOther = 96;
constexpr int kRegLaunch = 96;
static_assert(2 * kRegSoftmax + 2 * kRegDecode + kRegOther <= 5 * kRegLaunch, "more registers than the block has");

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;  // Q, K or V: 128 rows
  static constexpr int kOffQ = 0, kOffK = 2 * kTile, kOffV = kOffK + 2 * kTile, kOffScale = kOffV + 2 * kTile;
  static constexpr int kOffSums = kOffScale + kScaleRing * 64, kOffBar = kOffSums + 2 * 128 * 8;
  static constexpr int kBars = 512, kSmem = kOffBar + kBars + 1024;  // 1024: alignment slack
  static constexpr int kColO = 256;                                  // tensor memory: S0, S1, then O0, O1
  static constexpr int kPW = D + kPartHead;                          // a partial
};

// A segment: rows r0 .. r0 + nrow - 1 (tokens x heads of a group) of request b for head h over position tiles j0 .. j1 - 1.
struct Segment {
  int b, row0, n, kv, r0, nrow, h, j0, j1;  // b < 0: no more
  __device__ __forceinline__ bool halves() const { return nrow > 128; }  // two tiles of rows; else positions by turns
  __device__ __forceinline__ int tiles() const { return halves() ? 2 : min(2, j1 - j0); }
};

template <int N>
struct Cursor {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, parity ^= 1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const AttnPagedParams p, const Split sp) {
  using C = Cfg<D>;
  constexpr int NJ = D / 32;
  extern __shared__ uint8_t tree_smem[];
  const uint32_t raw = smem_u32(tree_smem);
  uint8_t* sm = tree_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ __align__(16) int4 work[kWorks][3];
  __shared__ uint32_t tmem_slot;
  auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;

  const uint32_t bar = sm32 + C::kOffBar;
  const uint32_t s_full = bar, o_full = bar + 16, turn = bar + 32, p_full = bar + 48, p_most = bar + 64, k_full = bar + 96, k_empty = bar + 112, v_full = bar + 128,
                 v_empty = bar + 144, q_full = bar + 160, q_empty = bar + 176, sc_full = bar + 192, work_full = sc_full + 8 * kScaleRing,
                 work_empty = work_full + 8 * kWorks, drained = work_empty + 8 * kWorks,
                 sums_put = drained + 8, sums_used = sums_put + 16;
  static_assert(192 + 8 * kScaleRing + 16 * kWorks + 40 <= C::kBars, "barriers");
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(turn + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);  // (a lane of each warp)
      mbar_init(p_most + 8 * i, 4);
      mbar_init(k_full + 8 * i, 4);
      mbar_init(v_full + 8 * i, 4);
      mbar_init(k_empty + 8 * i, 2);  // both issuing warps: they follow every tile
      mbar_init(v_empty + 8 * i, 2);
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 2);
      mbar_init(sums_put + 8 * i, 4);
      mbar_init(sums_used + 8 * i, 4);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full + 8 * i, 4);
    for (int i = 0; i < kWorks; ++i) {
      mbar_init(work_full + 8 * i, 1);
      mbar_init(work_empty + 8 * i, 8 + 8 + 2 + 1);  // the warps of softmax, decoding, issue and the second one ahead
    }
    mbar_init(drained, 2);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_serve();  // (all but the sums and the query rows is set up beside the kernel that makes those)
  float4* scales = reinterpret_cast<float4*>(sm + C::kOffScale);  // [ring][kf, f, 2^-f, mask][4 groups]
  bool ok = true;
  auto arrive = [&](uint32_t b) {  // of a whole warp: what its lanes did before is done
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  auto as_segment = [&](const int4 (&w)[3]) {
    Segment s;
    s.b = uni(w[0].x), s.row0 = uni(w[0].y), s.n = uni(w[0].z), s.kv = uni(w[0].w);
    s.r0 = uni(w[1].x), s.nrow = uni(w[1].y), s.h = uni(w[1].z), s.j0 = uni(w[1].w), s.j1 = uni(w[2].x);
    return s;
  };
  // The k-th segment, for a whole warp; b < 0 behind the last one, or where the wait ran out.
  auto take = [&](uint32_t k) {
    const int slot = k % kWorks;
    int4 w[3] = {make_int4(-1, 0, 0, 0), make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
    if (all_wait(work_full + 8 * slot, (k / kWorks) & 1)) {
#pragma unroll
      for (int i = 0; i < 3; ++i) w[i] = work[slot][i];
    } else {
      ok = false;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(work_empty + 8 * slot);
    return as_segment(w);
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax: one row per thread
    regs_up<kRegSoftmax>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    float2* sums = reinterpret_cast<float2*>(sm + C::kOffSums);  // [tile][row]: max, sum
    uint32_t mine_done = 0, all_done = 0, ends = 0, merges = 0;
    for (uint32_t k = 0; ok; ++k) {
      const Segment w = take(k);
      if (w.b < 0) break;
      const bool halves = w.halves();
      const int first_row = halves ? 128 * t : 0, r = w.r0 + first_row + row, active = w.tiles();
      const bool idle = first_row + 32 * (warp & 3) >= w.nrow;  // no row of the warp is there
      const bool there = first_row + row < w.nrow;              // (rows that are not hold anything)
      const int tok = min(r / p.G, w.n - 1), fresh = w.kv - w.n;  // positions before `fresh` are seen by every row
      const uint32_t* mask_row = p.mask + (int64_t)(w.row0 + tok) * p.mask_stride;
      float m = -INFINITY, l = 0.0f;
      bool begun = false;
      const int step = halves ? 1 : 2;
      for (int j = w.j0 + (halves ? 0 : t); j < w.j1; j += step, ++mine_done) {
        const uint32_t seq = all_done + (j - w.j0);
        if (!all_wait(s_full + 8 * t, mine_done & 1) || !all_wait(sc_full + 8 * (seq % kScaleRing), (seq / kScaleRing) & 1)) {
          ok = false;
          break;
        }
        fence_after();
        if (idle) {
          arrive(p_most + 8 * t);
          arrive(p_full + 8 * t);
          continue;
        }
        const float* sc = reinterpret_cast<const float*>(scales + 4 * (seq % kScaleRing));  // kf, f, 2^-f, mask of the four groups
        const uint4 exist = reinterpret_cast<const uint4*>(sc)[3];
        // Code is short here on purpose, in loops: what four kinds of warps run side by side has to stay in the
        // instruction caches (unrolled, a third of all issue slots went by without an instruction).
        const uint32_t s_at = tmem + lane_base + 128 * t;
        uint32_t s[2][32];
        // a tile with new tokens, or with positions behind the end or on a page outside the pool: hidden scores become -infinity
        if (kKeys * j + kKeys > fresh || (exist.x & exist.y & exist.z & exist.w) != 0xFFFFFFFFu) {
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            uint32_t bits = g == 0 ? exist.x : g == 1 ? exist.y : g == 2 ? exist.z : exist.w;
            const int at = kKeys * j + 32 * g - fresh;  // the group's first position among the new tokens
            if (at > -32) {
              uint32_t seen = tree_bits(mask_row, at, w.n);
              if (at < 0) seen |= (1u << -at) - 1u;  // the history
              bits &= seen;
            }
            tmem_ld32(s_at + 32 * g, s[0]);
            wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) s[0][c] = ((bits >> c) & 1u) ? s[0][c] : 0xFF800000u;
            tmem_st32(s_at + 32 * g, s[0]);
          }
          wait_st();
        }
        // The scores are read twice, for the maximum and for the weights, 32 at a time and 32 ahead: a thread that kept
        // them all would take the registers of the second warpgroup that decodes.
        tmem_ld32(s_at, s[0]);
        float mx = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < 4; g += 2) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            wait_ld();
            tmem_ld32(s_at + 32 * ((g + x + 1) & 3), s[x ^ 1]);
            float q[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 4)
#pragma unroll
              for (int i = 0; i < 2; ++i) q[i] = max3(q[i], __uint_as_float(s[x][c + 2 * i]), __uint_as_float(s[x][c + 2 * i + 1]));
            mx = fmaxf(mx, fmaf(fmaxf(q[0], q[1]), sc[g + x], sc[4 + g + x]));
          }
        }
        const bool need = mx > m + kPLazy && there;
        if (__any_sync(0xffffffffu, need)) {
          const float to = need ? mx : m;
          const float fac = to == m ? 1.0f : ex2(m - to);
          m = to;
          if (begun) {
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
        begun = true;
        const float up = kPBias - (m == -INFINITY ? 0.0f : m);
#pragma unroll 1
        for (int g = 0; g < 4; g += 2) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            wait_ld();
            if (x == 0 || g == 0) tmem_ld32(s_at + 32 * (g + x + 1), s[x ^ 1]);
            const float kf = sc[g + x], uf = up + sc[4 + g + x];
            const f32x2 kf2(kf, kf), u2(uf, uf);
            f32x2 sum[2] = {f32x2(0.0f, 0.0f), f32x2(0.0f, 0.0f)};
            uint32_t o[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float x0, x1;
              fma2(f32x2(__uint_as_float(s[x][c]), __uint_as_float(s[x][c + 1])), kf2, u2).get(x0, x1);
              x0 = ex2(x0), x1 = ex2(x1);
              sum[(c / 2) & 1] = add2(sum[(c / 2) & 1], f32x2(x0, x1));
              const __half2 hv = __floats2half2_rn(x0, x1);
              o[c / 2] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            float a, c;
            add2(sum[0], sum[1]).get(a, c);
            l = fmaf(a + c, sc[8 + g + x], l);
            tmem_st16(s_at + 16 * (g + x), o);
            if (x == 0 && g == 2) {  // three quarters of P are handed over while the last one is made
              wait_st();
              fence_before();
              arrive(p_most + 8 * t);
            }
          }
        }
        wait_st();
        fence_before();
        arrive(p_full + 8 * t);
      }
      all_done += w.j1 - w.j0;
      // ---- this segment's maximum, sum and O for the joining kernel
      if (t >= active) continue;
      if (ok && !all_wait(o_full + 8 * t, ends & 1)) ok = false;
      ++ends;
      // positions by turns: the two tiles' sums are of the same rows; each warpgroup adds up half of the channels
      const bool both = !halves && active == 2;
      {
        float f[2] = {1.0f, 1.0f}, M = m, L = l;
        if (both) {
          sums[128 * t + row] = make_float2(m, l);
          fence_after();
          fence_before();
          arrive(sums_put + 8 * t);
          if (!all_wait(sums_put + 8 * (t ^ 1), merges & 1)) ok = false;
          const float2 x = sums[row], y = sums[128 + row];
          M = fmaxf(x.x, y.x);
          f[0] = x.x == M ? 1.0f : ex2(x.x - M), f[1] = y.x == M ? 1.0f : ex2(y.x - M);
          L = fmaf(f[0], x.y, f[1] * y.y);
        }
        fence_after();
        const int c0 = both ? D / 2 * t : 0, c1 = both ? c0 + D / 2 : D;
        if (ok && !idle) {
          const int rb = first_row + row;  // row of the block
          float* dst = w.j0 > 0 ? sp.more + ((int64_t)blockIdx.x * kRows + rb) * C::kPW
                                : sp.first + ((int64_t)(w.h * p.total_q + w.row0) * p.G + r) * C::kPW;
          if (there && c0 == 0) *reinterpret_cast<float2*>(dst + 4) = make_float2(M, L);
#pragma unroll 1
          for (int c = c0; c < c1; c += 16) {
            uint32_t a[16];
            tmem_ld16(tmem + lane_base + C::kColO + (both ? 0 : D * t) + c, a);
            if (both) {
              uint32_t b[16];
              tmem_ld16(tmem + lane_base + C::kColO + D + c, b);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) a[i] = __float_as_uint(fmaf(__uint_as_float(a[i]), f[0], __uint_as_float(b[i]) * f[1]));
            } else {
              wait_ld();
            }
            if (there) {
              st_global_v8(dst + 8 + c, a);
              st_global_v8(dst + 8 + c + 8, a + 8);
            }
          }
        }
        fence_before();
        if (both) {  // the other warpgroup has read this one's O and sums before they are written again
          arrive(sums_used + 8 * t);
          if (!all_wait(sums_used + 8 * (t ^ 1), merges & 1)) ok = false;
          fence_after();
          ++merges;
        }
      }
    }
  } else if (warp < kAheadWarp) {
    // ------------------------------------------------------------ decode K, decode V: a warpgroup each
    // Two warps of a scheduler decode the same (K on the first two schedulers): half the code beside the softmax's.
    const int w4 = (warp & 1) + ((warp >> 1) & 2);  // positions 32 w4 .. 32 w4 + 31 of each tile
    const uint32_t page_bytes = (uint32_t)p.L.nkv * p.L.block;
    // The tiles of all segments one after the other: `ahead` is the one whose pages are looked up, `next` the one whose
    // bytes are loaded while `now` is decoded.  Scales and pages belong to position `lane` of the warp's.
    struct Tile {
      int b, kv, h, j, j1;
    } ahead = {-1, 0, 0, 0, 0}, next = ahead, now = ahead;
    uint32_t taken = 0;
    auto step = [&] {
      if (ahead.j + 1 < ahead.j1) {
        ++ahead.j;
      } else if (taken == 0 || ahead.b >= 0) {
        const Segment s = take(taken++);
        ahead = {s.b, s.b < 0 ? 0 : s.kv, s.h, s.j0, s.j1};
      }
    };
    int page_next = -1, page = 0;
    bool there = false, there_next = false;
    uint32_t sc = 0u, sc_next = 0u;
    // (tables, masks and pages as constants: see tree_prepare_kernel)
    auto look_up = [&] {  // the pages of the tile behind `next` (raw entries; positions behind the end, and no tile: -1)
      step();
      const int pos = kKeys * ahead.j + 32 * w4 + lane;
      page_next = ahead.b >= 0 && pos < ahead.kv ? __ldg(p.table + (int64_t)ahead.b * p.table_stride + (pos >> p.L.pshift)) : -1;
    };
    // The bytes of a tile are loaded whatever its pages are (page 0's for those outside the pool, and behind the last
    // tile): loads under a condition would be waited for where they stand.
    auto begin = [&] {
      next = ahead;
      const int pos = kKeys * next.j + 32 * w4 + lane;
      there_next = pos < next.kv && (uint32_t)page_next < (uint32_t)p.L.npages;
      page = there_next ? page_next : 0;
      sc_next = ld_stream_u32(p.pages + (size_t)next.h * p.L.block + (uint64_t)(uint32_t)page * page_bytes + p.L.soff + 4 * (pos & (p.L.psize - 1)));
    };
    // the place of positions 16 q .. 16 q + 15 of the warp's, which are on one page
    auto place = [&](int q) {
      const int pg = __shfl_sync(0xffffffffu, page, 16 * q), pin = (kKeys * next.j + 32 * w4 + 16 * q) & (p.L.psize - 1);
      return p.pages + (size_t)next.h * p.L.block + (uint64_t)(uint32_t)pg * page_bytes + pin * (D / 2);
    };
    using Piece = typename std::conditional<D == 128, uint4, uint2>::type;
    auto load = [](const uint8_t* at) {
      if constexpr (D == 128) return ld_stream_v4(at);
      else return ld_stream_v2(at);
    };
    // An entry with a scale from 2^110 on, or one that is not finite, makes the rows that see it NaN, but must not reach
    // its neighbours, nor the rows that do not see it: its K operand is NaN, which is one column of S, masked like any
    // other, and its V operand is 0.
    auto is_poor = [&] { return (sc & 0x7FFFu) >= kTooLarge || ((sc >> 16) & 0x7FFFu) >= kTooLarge; };
    // The 32 positions' scales relative to their largest's power of two are multipliers of the decoded words (codes x
    // 2^-24 and, for odd values, x 2^-20): code x (scale / 2^e) x 2^-9, or x 2^-1 where a scale's exponent is more than
    // 7 below the largest's.
    auto wide_of = [&](uint32_t x, uint32_t& e) {
      e = __reduce_max_sync(0xffffffffu, x);
      return __any_sync(0xffffffffu, x != 0u && x + 7u < e);
    };
    regs_down<kRegDecode>();
    if ((warp & 2) == 0) {
      // piece (lane & 3) of positions 8 i + (lane >> 2): words of all j of one pair of columns
      // (lanes two pieces apart would store to the same banks of two panels: the second take their words in another order)
      Piece kw[4], kn[4];
      const int turn = D == 128 ? lane & 2 : 0;
      auto load_k = [&] {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* src = place(i / 2) + ((lane >> 2) + 8 * (i & 1)) * (D / 2) + (lane & 3) * (D / 8);
          if constexpr (D == 128) {
            const uint2 a = ld_stream_v2(src + 4 * turn), b = ld_stream_v2(src + 8 - 4 * turn);
            kn[i] = make_uint4(a.x, a.y, b.x, b.y);
          } else {
            kn[i] = load(src);
          }
        }
      };
      look_up();
      begin();
      load_k();
      look_up();
      for (uint32_t seq = 0; ok; ++seq) {
        const int st = seq & 1;
        const uint32_t use = seq >> 1;
        now = next, sc = sc_next, there = there_next;
#pragma unroll
        for (int i = 0; i < 4; ++i) kw[i] = kn[i];
        if (now.b < 0) break;
        begin();
        load_k();
        look_up();
        if (kKeys * now.j + 32 * w4 + lane < now.kv && !there) set_status(p.status, FT_DEV_RANGE);
        if (!there) sc = 0u;
        const bool poor = is_poor();
        if (poor) sc = 0u;
        uint32_t ek, ev;
        const bool wide_k = wide_of((sc & 0x7FFFu) >> 7, ek), wide_v = wide_of((sc >> 23) & 0xFFu, ev);
        ek = max(ek, 27u), ev = ev == 0u ? kNoScaleExp : max(ev, 27u);
        const float mk = poor ? __uint_as_float(0x7FC00000u) : __uint_as_float(sc << 16) * __uint_as_float((268u - ek) << 23);
        const __half2 mk2 = __floats2half2_rn(mk, mk * 0.0625f);  // (even, odd values)
        const uint32_t mku = *reinterpret_cast<const uint32_t*>(&mk2), exist = __ballot_sync(0xffffffffu, there);
        if (use > 0 && !all_wait(k_empty + 8 * st, (use - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          float* dst = reinterpret_cast<float*>(scales + 4 * (seq % kScaleRing)) + w4;
          const uint32_t tv = wide_v ? ev - 8u : ev;
          dst[0] = __uint_as_float((wide_k ? ek - 4u : ek + 4u) << 23);  // 2^(e + 9) / kQUp (or 2^-8 of it), e = ek - 126
          dst[4] = (float)((int)tv - 126);
          dst[8] = __uint_as_float((253u - tv) << 23);
          dst[12] = __uint_as_float(exist);
        }
        uint8_t* kd = sm + C::kOffK + st * C::kTile;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * w4 + 8 * i + (lane >> 2);
          const uint32_t both = __shfl_sync(0xffffffffu, mku, 8 * i + (lane >> 2));
          const uint32_t m0 = prmt(both, both, 0x1010u), m1 = prmt(both, both, 0x3232u);
          const uint32_t* x = reinterpret_cast<const uint32_t*>(&kw[0]);
#pragma unroll
          for (int k = 0; k < NJ; ++k) {
            const int w = (lane & 3) * NJ + (k ^ turn);  // word of the entry: slots 8 w .. 8 w + 7 of the operand's row
            uint32_t r[4];
            paged_word(x[k], r);
            if (wide_k) {
#pragma unroll
              for (int e = 0; e < 4; ++e) r[e] = hmul2(r[e], kWide);
            }
            *reinterpret_cast<uint4*>(kd + (w / 8) * (kKeys * 128) + key * 128 + (((w % 8) ^ (key & 7)) << 4)) =
                make_uint4(hmul2(r[0], m0), hmul2(r[1], m1), hmul2(r[2], m0), hmul2(r[3], m1));
          }
          kw[0] = kw[1], kw[1] = kw[2], kw[2] = kw[3];
        }
        fence_proxy_async_smem();
        arrive(sc_full + 8 * (seq % kScaleRing));
        arrive(k_full + 8 * st);
      }
    } else {
      // chunk (lane & 7) of pairs 4 (lane >> 3) + k: words of all j for eight positions
      Piece vw[4], vn[4];
      const int g = lane & 7, grp = lane >> 3;
      auto load_v = [&] {
        const uint8_t *lo = place(0), *hi = place(1), *src = ((grp & 2) ? hi : lo) + p.L.voff + (grp & 1) * 4 * D;
#pragma unroll
        for (int k = 0; k < 4; ++k) vn[k] = load(src + k * D + (g ^ paged_v_turn<D>(k)) * (D / 8));
      };
      look_up();
      begin();
      load_v();
      look_up();
      for (uint32_t seq = 0; ok; ++seq) {
        const int st = seq & 1;
        const uint32_t use = seq >> 1;
        now = next, sc = sc_next, there = there_next;
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = vn[i];
        if (now.b < 0) break;
        begin();
        load_v();
        look_up();
        if (!there || is_poor()) sc = 0u;
        uint32_t ev;
        const bool wide_v = wide_of((sc >> 23) & 0xFFu, ev);
        ev = ev == 0u ? kNoScaleExp : max(ev, 27u);
        const float mv = __uint_as_float(sc & 0xFFFF0000u) * __uint_as_float((268u - ev) << 23);
        const float mv_next = __shfl_down_sync(0xffffffffu, mv, 1);
        const __half2 mv2 = __floats2half2_rn(mv, mv_next);  // at even lanes: a pair of positions
        const uint32_t mvu = *reinterpret_cast<const uint32_t*>(&mv2);
        uint32_t m0[4], m1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m0[k] = __shfl_sync(0xffffffffu, mvu, 8 * grp + 2 * k);
          m1[k] = hmul2(m0[k], 0x2C002C00u);  // / 16
        }
        if (use > 0 && !all_wait(v_empty + 8 * st, (use - 1) & 1)) {
          ok = false;
          break;
        }
        const int chunk = 4 * w4 + grp;  // 8 positions
        uint8_t* panel = sm + C::kOffV + st * C::kTile + (chunk / 8) * (D * 128);
#pragma unroll 1
        for (int j = 0; j < NJ; ++j) {
          uint32_t r[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            paged_word(vw[k].x, r[k]);
            if (wide_v) {
#pragma unroll
              for (int e = 0; e < 4; ++e) r[k][e] = hmul2(r[k][e], kWide);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) r[k][e] = hmul2(r[k][e], (e & 1) ? m1[k] : m0[k]);
            vw[k].x = vw[k].y;
            if constexpr (D == 128) vw[k].y = vw[k].z, vw[k].z = vw[k].w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = 32 * j + g + 8 * e;
            *reinterpret_cast<uint4*>(panel + ch * 128 + (((chunk % 8) ^ (ch & 7)) << 4)) = make_uint4(r[0][e], r[1][e], r[2][e], r[3][e]);
          }
        }
        fence_proxy_async_smem();
        arrive(v_full + 8 * st);
      }
    }
  } else {
    regs_down<kRegOther>();
    if (warp >= kMmaWarp) {
      // ---------------------------------------------------------- tensor-core issue, a warp for each tile
      constexpr uint32_t id_qk = idesc_f16(128, kKeys), id_pv = idesc_f16(128, D);
      const uint32_t lead = lane == 0 ? 1u : 0u, tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int t = warp - kMmaWarp;
      const uint32_t q_lo = desc_lo(sm32 + C::kOffQ), k_lo = desc_lo(sm32 + C::kOffK), v_lo = desc_lo(sm32 + C::kOffV);
      const uint32_t ds = tm + 128 * t, d_o = tm + C::kColO + D * t;
      Cursor<2> q_at;  // the segment's first query tile
      uint32_t seq0 = 0, mine_done = 0, turns_done = 0;
      auto full = [&](uint32_t at, uint32_t seq) { return all_wait(at + 8 * (seq & 1), (seq >> 1) & 1); };
      for (uint32_t k = 0; ok; ++k) {
        const Segment w = take(k);
        if (w.b < 0) break;
        const bool halves = w.halves();
        const int count = w.j1 - w.j0, step = halves ? 1 : 2, first = halves ? 0 : t;
        const uint32_t qa = q_lo + (halves ? q_at.slot ^ t : q_at.slot) * (C::kTile >> 4);
        const bool turns = w.tiles() == 2;
        auto qk = [&](int i, auto&& pass) {
          const uint32_t ka = k_lo + ((seq0 + i) & 1) * (C::kTile >> 4);
          mma_ss<false>(ds, qa, ka, id_qk, lead);
#pragma unroll
          for (int ks = 1; ks < D / 16; ++ks) {
            const uint32_t o = ((ks / 4) * (128 * 128) + 32 * (ks % 4)) >> 4;
            if (ks == D / 16 - 1) pass();
            mma_ss<true>(ds, qa + o, ka + o, id_qk, lead);
          }
          commit(s_full + 8 * t, lead);
          commit(k_empty + 8 * ((seq0 + i) & 1), lead);
        };
        auto pv = [&](int i, int from, int to) {
          const uint32_t va = v_lo + ((seq0 + i) & 1) * (C::kTile >> 4);
#pragma unroll
          for (int ks = from; ks < to; ++ks)
            mma_ts(d_o, ds + 8 * ks, va + (((ks / 4) * (D * 128) + 32 * (ks % 4)) >> 4), id_pv, ks > 0 || i != first ? 1u : 0u, lead);
        };
        // The tiles take the tensor core by turns, tile 0 first.
        auto pass = [&] {
          if (turns && lead) mbar_arrive(turn + 8 * (t ^ 1));
        };
        auto my_turn = [&] {
          if (!turns) return true;
          const uint32_t i = turns_done++;
          return t == 0 ? i == 0 || all_wait(turn, (i - 1) & 1) : all_wait(turn + 8, i & 1);
        };
        // tile i of the other's K or V: followed, so that no use of a place is missed
        auto follow = [&](uint32_t there, uint32_t empty, int i) {
          if (!full(there, seq0 + i)) return false;
          if (lead) mbar_arrive(empty + 8 * ((seq0 + i) & 1));
          return true;
        };
        // the query tiles: both (halves), or the one that both tiles share
        {
          Cursor<2> q = q_at;
          for (int i = 0; ok && i < (halves ? 2 : 1); ++i, q.next()) ok = all_wait(q_full + 8 * q.slot, q.parity);
        }
        if (!ok) break;
        int rounds = 0;  // batches of the tile with more of them: both go through as many turns
        const int most = halves ? count : (count + 1) / 2;
        if (ok && first < count) {
          ok = (first == 0 || halves || follow(k_full, k_empty, 0)) && full(k_full, seq0 + first);
          if (!ok) break;
          fence_after();
          qk(first, [] {});
          for (int i = first; ok && i < count; i += step, ++mine_done, ++rounds) {
            // all that can be waited for outside of the turn
            const bool more = i + step < count;
            ok = (halves || i == 0 || follow(v_full, v_empty, i - 1)) && full(v_full, seq0 + i) &&
                 (!more || ((halves || follow(k_full, k_empty, i + 1)) && full(k_full, seq0 + i + step))) &&
                 all_wait(p_most + 8 * t, mine_done & 1) && my_turn();
            if (!ok) break;
            fence_after();
            pv(i, 0, 6);
            ok = all_wait(p_full + 8 * t, mine_done & 1);
            if (!ok) break;
            fence_after();
            pv(i, 6, 8);
            commit(v_empty + 8 * ((seq0 + i) & 1), lead);
            if (more) {
              qk(i + step, pass);
            } else {
              commit(o_full + 8 * t, lead);
              pass();
              if (!halves && i + 1 < count) ok = follow(k_full, k_empty, i + 1) && follow(v_full, v_empty, i + 1);
            }
          }
        } else if (ok) {  // (one tile of positions: the other's)
          ok = follow(k_full, k_empty, 0) && follow(v_full, v_empty, 0);
        }
        for (; ok && turns && rounds < most; ++rounds) {
          ok = my_turn();
          pass();
        }
        // (every product of this segment that reads the query tiles is issued)
        for (int i = 0; i < (halves ? 2 : 1); ++i, q_at.next()) commit(q_empty + 8 * q_at.slot, lead);
        seq0 += count;
      }
      // tensor memory is freed only when nothing issued here is in flight
      commit(drained, lead);
      if (!all_wait(drained, 0)) ok = false;
    } else if (warp == kAheadWarp) {
      // ---------------------------------------------------------- segments
      Share share;
      share.begin(p, sp, lane);
      for (uint32_t k = 0; ok; ++k) {
        Segment w = {};
        int block = 0;
        w.b = -1;
        if (share.next(p, sp, block, w.h, w.j0, w.j1)) {
          w.b = share.b, w.row0 = share.req.y, w.n = share.req.z, w.kv = share.req.w;
          w.r0 = block * kRows, w.nrow = min(w.n * p.G - w.r0, kRows);
        }
        if (k >= kWorks && !all_wait(work_empty + 8 * (k % kWorks), (k / kWorks - 1) & 1)) ok = false;
        if (ok && lane == 0) {
          work[k % kWorks][0] = make_int4(w.b, w.row0, w.n, w.kv);
          work[k % kWorks][1] = make_int4(w.r0, w.nrow, w.h, w.j0);
          work[k % kWorks][2] = make_int4(w.j1, 0, 0, 0);
          mbar_arrive(work_full + 8 * (k % kWorks));
        }
        if (w.b < 0) break;
      }
    } else {
      // ---------------------------------------------------------- query rows: 16-byte chunks to their places in the operand
      // (rows behind the last one stay as they are: nobody looks at what comes of them)
      constexpr int kChunks = D / 8;
      Cursor<2> q_at;
      uint32_t q_used = 0;
      for (uint32_t k = 0; ok; ++k) {
        const Segment w = take(k);
        if (w.b < 0) break;
        for (int t = 0; t < (w.halves() ? 2 : 1); ++t, q_at.next(), ++q_used) {
          if (q_used >= 2 && !all_wait(q_empty + 8 * q_at.slot, q_at.parity ^ 1)) {
            ok = false;
            break;
          }
          const uint32_t to = sm32 + C::kOffQ + q_at.slot * C::kTile;
          const int rows = min(128, w.nrow - 128 * t), c = lane % kChunks;
          const uint16_t* from = sp.q + ((int64_t)(w.h * p.total_q + w.row0) * p.G + w.r0 + 128 * t) * D + 8 * c;
#pragma unroll 4
          for (int r = lane / kChunks; r < rows; r += 32 / kChunks) cp_async16(to + chunk_at(128, r, c), from + (int64_t)r * D);
          cp_async_wait_all();
          fence_proxy_async_smem();
          arrive(q_full + 8 * q_at.slot);
        }
      }
    }
  }
  if (!ok) set_status(p.status, FT_DEV_TIMEOUT);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

template <int D>
static cudaError_t launch(const AttnPagedParams& p, void* workspace, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    // the roles' register shares add up to kRegLaunch a thread: a build with fewer would wait for them forever
    cudaFuncAttributes fa = {};
    if (cudaFuncGetAttributes(&fa, tree_kernel<D>) != cudaSuccess) return cudaErrorInvalidDeviceFunction;
    if (fa.numRegs < kRegLaunch) return cudaErrorInvalidConfiguration;
    allowed[dev] = 1;
  }
  Split sp = split_of(workspace, p.B, (int64_t)p.total_q * p.L.nkv * p.G, D, num_sms(), kRows);
  sp.seg = kSegUnits;
  sp.odd = 1.0f, sp.up = kOScale;
  cudaError_t e = launch_prepare<D>(p, sp, st);
  if (e != cudaSuccess) return e;
  e = launch_served(tree_kernel<D>, dim3((unsigned)sp.ctas), dim3(kThreads), Cfg<D>::kSmem, st, 1, p, sp);
  return e != cudaSuccess ? e : launch_join<D>(p, sp, st);
}

}  // namespace tree

size_t attn_tree_ws(int nkv, int G, int head_dim, int B, int total_q) {
  return tree::split_bytes(B, (int64_t)total_q * nkv * G, head_dim, tree::num_sms(), tree::kRows);
}

bool attn_tree_fits(const AttnPagedParams& p) {
  return tree::units_fit(p);
}

cudaError_t launch_attn_tree(const AttnPagedParams& p, int head_dim, void* workspace, cudaStream_t st) {
  return head_dim == 128 ? tree::launch<128>(p, workspace, st) : tree::launch<64>(p, workspace, st);
}

}  // namespace ft
