// Attention of small draft trees (17 to 32 rows, tokens x heads of a group) over the paged 4-bit cache, on the
// fifth-generation tensor cores with the positions as the products' rows:
//   S^T = K Q^T     A = K codes from tensor memory (128 positions), B = the query rows from shared memory (N = 32)
//   O^T += V^T P^T  A = V codes from tensor memory (the channels), B = P from shared memory
// so that a thread has one position's scores of all rows: the position's scales are two of its registers, the codes need
// no scale, and as an FP16 subnormal each costs 7 instructions for eight of them.  What a row of products with 128 of them
// would do for rows that are not there is left out, and shared memory holds 16 KB of operands where it held 160.
// How the work is shared out and joined: ft_attn_tree.cuh; the arithmetic: that of the kernel for few rows in
// ft_attn_paged.cu.
//
// A CTA has eight warps that work (two threads a position: half of the channels of K, half of the rows of the softmax; V
// by words) and one that issues; two CTAs an SM, whose phases fill each other's waits:
//   tile i: K decoded (while P V of tile i - 1 runs), V decoded (while Q K^T runs), softmax
// Bytes come by 16-byte asynchronous copies, a tile ahead.  The running max moves when a score passes it by 2^4.
// A tile's maxima go through shared memory, a row to eight threads: 32 reductions of a warp took 2000 cycles and, being
// straight code that runs once a segment, their fetching from a cold instruction cache 7000 in a first tile.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
//
// Measured, 32 requests of up to 4096 positions, 7 tokens (28 rows) of 32 heads over 8: 45 us of the call's three kernels
// (65 MB, 1459 GB/s), of which 5 are the kernel before and 8 the joining one; lengths of 64: 23.  Neither the issue slots
// (45%) nor HBM (22%) are at their end: what bounds it is the chain of a tile, 535 instructions a warp of which a third
// decode, with two CTAs an SM to cover it (26% of the warps resident; 96 registers, 40 bytes of them spilled).  With four
// working warps it was 52 and 60.
#include "ft_attn_tree.cuh"

namespace ft {

namespace tree {

namespace few {

constexpr int kWork = 256, kThreads = kWork + 32, kMaxRows = 32, kPerSm = 2;
constexpr int kSegUnits = 3;  // a segment's cost beside its positions, in tiles of them

template <int D>
struct Cfg {
  static constexpr int kStage = kKeys * D;  // K and V of a tile, as they are
  static constexpr int kPitch = D + 8;      // of O's rows on their way out
  static constexpr int kOffQ = 0, kOffP = kMaxRows * D * 2, kOffRing = kOffP + kKeys * kMaxRows * 2;
  static constexpr int kOffX = kOffRing + 2 * kStage, kOffRows = kOffX + kKeys * kMaxRows * 4;
  static constexpr int kOffBar = kOffRows + 5 * kMaxRows * 4;
  static_assert(kMaxRows * kPitch * 4 <= 2 * kStage, "O in the ring");
  static constexpr int kSmem = 100 * 1024;  // (more than it takes: no third CTA of an SM, which would wait for tensor memory)
  static_assert(kOffBar + 64 + 1024 <= kSmem, "shared memory");
  static constexpr int kColK = 0, kColV = 64, kColS = 128, kColO = 160, kCols = 256;  // tensor memory
};

// B = P, 32 rows contiguous for each position: 64-byte swizzle, MN-major, groups of 8 positions 512 bytes apart.
constexpr uint32_t kDescHiP = (512u >> 4) | (1u << 14) | (4u << 29);
__device__ __forceinline__ void mma_ts_p(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 y; mov.b64 y, {%2, %4}; setp.ne.u32 p, %5, 0;\n"
      "setp.ne.u32 e, %6, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHiP), "r"(acc), "r"(lead)
      : "memory");
}
// 16 lanes x 32 columns from the fragments of products of 16 rows (a lane: two columns of each eight, of rows lane / 4 and + 8).
__device__ __forceinline__ void tmem_st16x256b(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Whether any of the working threads says so.
__device__ __forceinline__ bool any_of_work(bool x) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 1, 256, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"((uint32_t)x)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ void work_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) tree_few_kernel(const AttnPagedParams p, const Split sp) {
  using C = Cfg<D>;
  constexpr int CE = D / 32;  // 16-byte chunks of a K entry
  extern __shared__ uint8_t few_tree_smem[];
  const uint32_t raw = smem_u32(few_tree_smem);
  uint8_t* sm = few_tree_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ int4 seg[2][2];
  __shared__ int failed;
  __shared__ uint32_t tmem_slot;
  float *row_m = reinterpret_cast<float*>(sm + C::kOffRows), *row_u = row_m + kMaxRows;  // running max, kPBias - max (kPBias for none yet)
  float *row_fac = row_u + kMaxRows, *row_up = row_fac + kMaxRows;                       // at its last move: factor of the sums, change of row_u
  uint32_t* seen_by = reinterpret_cast<uint32_t*>(row_up + kMaxRows);                    // the rows that see a new token
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  const uint32_t bar = sm32 + C::kOffBar, k_put = bar, s_full = bar + 8, p_put = bar + 16, o_full = bar + 24;
  if (tid == 0) {
    mbar_init(k_put, kWork / 32);  // (a lane of each working warp)
    mbar_init(p_put, kWork / 32);
    mbar_init(s_full, 1);
    mbar_init(o_full, 1);
    mbar_fence_init();
    failed = 0;
  }
  if (warp == kWork / 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "n"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_serve();  // (all but the sums and the query rows is set up beside the kernel that makes those)
  bool ok = true;
  auto arrive = [&](uint32_t b) {  // of a whole warp: what its lanes did before is done
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };

  // ---- this CTA's share: the issuing warp works out a segment while the one before it is worked on
  Share share;
  auto find = [&](int to) {
    int block, h, j0, j1;
    const bool found = share.next(p, sp, block, h, j0, j1);
    if (lane == 0) {
      seg[to][0] = make_int4(found ? share.b : -1, share.req.y, share.req.z, share.req.w);
      seg[to][1] = make_int4(h, j0, j1, 0);
    }
  };
  if (warp == kWork / 32) {
    share.begin(p, sp, lane);
    find(0);
  }
  __syncthreads();
  uint32_t done = 0;  // tiles of the segments before this one
  for (int turn = 0;; turn ^= 1) {
    const int4 s0 = seg[turn][0], s1 = seg[turn][1];
    if (s0.x < 0) break;
    const int s_b = s0.x, s_row0 = s0.y, s_n = s0.z, s_kv = s0.w, h = s1.x, j0 = s1.y, count = s1.z - s1.y;
    const int nrow = s_n * p.G;
    if (warp == kWork / 32) {
      // ------------------------------------------------------------ issue
      constexpr uint32_t id_qk = idesc_f16(128, kMaxRows), id_pv = idesc_f16(128, kMaxRows) | (1u << 16);  // (P is MN-major)
      const uint32_t lead = lane == 0 ? 1u : 0u, tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = desc_lo(sm32 + C::kOffQ), p_lo = desc_lo(sm32 + C::kOffP);
      for (int i = 0; i < count; ++i) {
        const uint32_t parity = (done + i) & 1;
        if (!all_wait(k_put, parity)) {
          ok = false;
          break;
        }
        fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ts(tm + C::kColS, tm + C::kColK + 8 * ks, q_lo + (((ks / 4) * (kMaxRows * 128) + 32 * (ks % 4)) >> 4), id_qk, ks > 0 ? 1u : 0u, lead);
        commit(s_full, lead);
        if (!all_wait(p_put, parity)) {
          ok = false;
          break;
        }
        fence_after();
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_ts_p(tm + C::kColO, tm + C::kColV + 8 * ks, p_lo + ((ks * 1024) >> 4), id_pv, ks > 0 || i > 0 ? 1u : 0u, lead);
        commit(o_full, lead);
      }
      find(turn ^ 1);
    } else {
      // ------------------------------------------------------------ work
      // a position's and a channel's work is two threads': `half` of its channels, positions or rows
      const int half = tid >> 7, t = tid & 127, w = warp & 3;
      const uint32_t lanes = (uint32_t)(32 * w) << 16;
      const int* table = p.table + (int64_t)s_b * p.table_stride;
      const int fresh = s_kv - s_n;  // positions before this one are seen by every row
      const uint64_t page_bytes = (uint64_t)((uint32_t)p.L.nkv * p.L.block);
      const uint8_t* base = p.pages + (size_t)h * p.L.block;
      const int64_t q_row = (int64_t)(h * p.total_q + s_row0) * p.G;
#pragma unroll
      for (int i = tid; i < kMaxRows * (D / 8); i += kWork) {  // query rows (zeros behind the last)
        const int r = i / (D / 8), c = i % (D / 8);
        cp_async16_zfill(sm32 + C::kOffQ + chunk_at(kMaxRows, r, c), sp.q + (q_row + min(r, nrow - 1)) * D + 8 * c, r < nrow);
      }
      if (tid < kMaxRows) row_m[tid] = -INFINITY, row_u[tid] = kPBias;
      // The bytes of tile i, K by one half, V by the other, 16 threads for each 16 positions, which are on one page: K entries
      // (chunks turned so that 8 lanes' reads meet 8 banks), V as it is; pages outside the pool and behind the end are page 0
      // (no scale, and hidden).  Pages are looked up a tile further ahead.  (Tables and pages as constants: see
      // tree_prepare_kernel.)
      const int grp = t >> 4, in = t & 15;
      const uint32_t ring = sm32 + C::kOffRing + grp * (16 * D / 2) + half * (kKeys * D / 2);
      const uint32_t even = ring + (D == 128 && half == 0 ? (in >> 2) * 64 + (((in & 3) ^ (in >> 3)) << 4) : 16 * in);
      const uint32_t odd = D == 128 && half == 0 ? even ^ 32 : even;
      int page = -1;
      auto look_up = [&](int i) {
        const int pos = kKeys * (j0 + i) + t;
        page = i < count && pos < s_kv ? __ldg(table + (pos >> p.L.pshift)) : -1;
      };
      uint32_t sc_next = 0u;
      bool there_next = false;
      auto copy = [&](int i) {
        const uint32_t st = (i & 1) * C::kStage;
        const int pos = kKeys * (j0 + i) + t;
        // (a group's first position is there if any of it is; its page is the one of all)
        const int first = __shfl_sync(0xffffffffu, page, lane & 16);
        const uint32_t at = (pos & ~15) & (p.L.psize - 1);
        const uint8_t* pg = base + ((uint32_t)first < (uint32_t)p.L.npages ? (uint32_t)first : 0u) * page_bytes;
        if (i < count) {
          const uint8_t* from = pg + (half ? p.L.voff : 0) + at * (D / 2) + 16 * in;
#pragma unroll
          for (int k = 0; k < CE; ++k) cp_async16(st + (k & 1 ? odd : even) + 256 * k, from + 256 * k);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        there_next = i < count && pos < s_kv && (uint32_t)page < (uint32_t)p.L.npages;
        if (i < count && pos < s_kv && !there_next) set_status(p.status, FT_DEV_RANGE);
        sc_next = ld_stream_u32(pg + p.L.soff + 4 * (at + in));
      };
      look_up(0);
      copy(0);
      look_up(1);
      if (warp == kWork / 32 - 1) {
        const uint32_t mask = lane < nrow ? p.mask[(int64_t)(s_row0 + lane / p.G) * p.mask_stride] : 0u;  // (up to 32 new tokens: one word)
        uint32_t mine = 0u;
#pragma unroll 4
        for (int a = 0; a < 32; ++a) {
          const uint32_t rows = __ballot_sync(0xffffffffu, (mask >> a) & 1u);
          mine = lane == a ? rows : mine;
        }
        seen_by[lane] = mine;
      }
      // Transposed through shared memory, rows of 32 floats by position: 8 threads a row take 16 positions each.
      float* X = reinterpret_cast<float*>(sm + C::kOffX);
      auto put = [&](int c, float a, float b, float d, float e) { *reinterpret_cast<float4*>(X + 32 * t + 4 * ((4 * half + c) ^ (t & 7))) = make_float4(a, b, d, e); };
      const int row = tid >> 3, eighth = tid & 7;
      auto get = [&](int k) {
        const int pos = 16 * eighth + ((k + eighth) & 15);
        return X[32 * pos + 4 * ((row >> 2) ^ (pos & 7)) + (row & 3)];
      };
      f32x2 l[8];  // this position's weights of each row, added up
#pragma unroll
      for (int r = 0; r < 8; ++r) l[r] = f32x2(0.0f, 0.0f);
      // words of V: chunk and place in it of word rho of a warp's eight
      auto word_g = [&](int rho) { return D == 128 ? 2 * w + (rho >> 2) : 4 * w + (rho >> 1); };
      auto word_j = [&](int rho) { return D == 128 ? rho & 3 : rho & 1; };
      int i = 0;
      for (; i < count; ++i) {
        const uint32_t parity = (done + i) & 1;
        const uint32_t sc = sc_next;
        const bool there = there_next;
        work_sync();  // the other stage's bytes have been read by all
        copy(i + 1);
        look_up(i + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        work_sync();
        const uint8_t* st = sm + C::kOffRing + (i & 1) * C::kStage;
        // ---- K: half of a position's channels (the operand's room is free: S of tile i - 1 was waited for)
        fence_after();
        {
          uint32_t x[D / 4];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const int ch = D / 64 * half + c;
            const uint4 q = *reinterpret_cast<const uint4*>(st + t * (D / 2) + 16 * (D == 128 ? ch ^ ((t >> 1) & 3) : ch));
            const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t r[4];
              paged_word(wd[k], r);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[16 * c + 4 * k + e] = r[e];
            }
          }
          if constexpr (D == 128) tmem_st32(tmem + lanes + C::kColK + 32 * half, x);
          else tmem_st16(tmem + lanes + C::kColK + 16 * half, x);
        }
        wait_st();
        if (i == 0) fence_proxy_async_smem();  // (the query rows)
        fence_before();
        arrive(k_put);
        // ---- V: half of the positions, when P V of tile i - 1 is through with the operands
        if (i > 0 && !all_wait(o_full, (done + i - 1) & 1)) ok = false;
        fence_after();
        // A word has 4 channels of a pair of positions.  Stored as 16 lanes x 256 bits, where a lane has two columns of row
        // lane / 4 and of row lane / 4 + 8, each word is read and decoded once: row 8 e + rho of a warp's is value e of word
        // rho, column 8 k + 2 q + s is pair 8 k + q + 4 s, and so 32 lanes read 32 banks.
        if (w < D / 32) {
          const int rho = lane >> 2, q = lane & 3;
          const uint8_t* v = st + kKeys * D / 2 + (32 * half + q) * D + (word_g(rho) ^ paged_v_turn<D>(q)) * (D / 8) + 4 * word_j(rho);
          uint32_t x[2][16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a[4], c[4];
            paged_word(*reinterpret_cast<const uint32_t*>(v + 8 * k * D), a);
            paged_word(*reinterpret_cast<const uint32_t*>(v + (8 * k + 4) * D), c);
#pragma unroll
            for (int y = 0; y < 2; ++y) x[y][4 * k] = a[2 * y], x[y][4 * k + 1] = c[2 * y], x[y][4 * k + 2] = a[2 * y + 1], x[y][4 * k + 3] = c[2 * y + 1];
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) tmem_st16x256b(tmem + lanes + ((uint32_t)(16 * y) << 16) + C::kColV + 32 * half, x[y]);
        }
        // ---- softmax: this thread's position, rows 16 half .. + 15
        const float ks = __uint_as_float(sc << 16) * kKsUp, vv = __uint_as_float(sc & 0xFFFF0000u);
        const float vs = vv == 0.0f ? kNoScale : fmaxf(vv, kMinScale);
        // (a scale from 2^110 on, kTooLarge, makes this and with it the scores NaN, whatever they were)
        const float lv = fmaf(fmaf(vv, kKsUp, ks), 0.0f, lg2(vs)), rs = there ? rcp(vs) : 0.0f;
        const int at = kKeys * (j0 + i) + t - fresh;  // the position among the new tokens
        if (!all_wait(s_full, parity)) ok = false;
        fence_after();
        uint32_t sr[16];
        tmem_ld16(tmem + lanes + C::kColS + 16 * half, sr);
        wait_ld();
        // x = s + kPBias - max, and whether it passes the bias by 2^4 (no max yet: kPBias)
        const f32x2 ks2(ks, ks), lv2(lv, lv);
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 u4 = *reinterpret_cast<const float4*>(row_u + 16 * half + r);
          fma2(f32x2(__uint_as_float(sr[r]), __uint_as_float(sr[r + 1])), ks2, add2(lv2, f32x2(u4.x, u4.y))).get(x[r], x[r + 1]);
          fma2(f32x2(__uint_as_float(sr[r + 2]), __uint_as_float(sr[r + 3])), ks2, add2(lv2, f32x2(u4.z, u4.w))).get(x[r + 2], x[r + 3]);
        }
        if (!__all_sync(0xffffffffu, there && at < 0)) {
          const uint32_t seen = (there ? at < 0 ? ~0u : seen_by[at & 31] : 0u) >> (16 * half);  // (at < n <= 32 where it is there)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[r] = (seen >> r) & 1u ? x[r] : -INFINITY;  // whatever the entry holds
        }
        float over = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; r += 2) over = max3(over, x[r], x[r + 1]);
        if (any_of_work(over > kPBias + kPLazy || i == 0 || !ok)) {
          if (any_of_work(!ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) put(c, x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          work_sync();
          float top = -INFINITY;
#pragma unroll 4
          for (int k = 0; k < 16; ++k) top = fmaxf(top, get(k));  // (passes over NaN)
          const float m_old = row_m[row], u_old = row_u[row];
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float m_new = fmaxf(top - u_old, m_old), u_new = kPBias - (m_new == -INFINITY ? 0.0f : m_new);
          if (eighth == 0) {
            row_m[row] = m_new, row_u[row] = u_new;
            row_fac[row] = m_old == m_new ? 1.0f : ex2(m_old - m_new);
            row_up[row] = u_new - u_old;
          }
          work_sync();
          if (i > 0) {
            uint32_t o[16];
            tmem_ld16(tmem + lanes + C::kColO + 16 * half, o);
            wait_ld();
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
              const float2 f = *reinterpret_cast<const float2*>(row_fac + 16 * half + r);
              o[r] = __float_as_uint(__uint_as_float(o[r]) * f.x), o[r + 1] = __float_as_uint(__uint_as_float(o[r + 1]) * f.y);
              l[r / 2] = mul2(l[r / 2], f32x2(f.x, f.y));
            }
            tmem_st16(tmem + lanes + C::kColO + 16 * half, o);
          }
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const float2 f = *reinterpret_cast<const float2*>(row_up + 16 * half + r);
            x[r] += f.x, x[r + 1] += f.y;
          }
        }
        uint32_t pr[8];
        const f32x2 rs2(rs, rs);
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const float x0 = ex2(x[r]), x1 = ex2(x[r + 1]);
          l[r / 2] = fma2(f32x2(x0, x1), rs2, l[r / 2]);
          const __half2 a = __floats2half2_rn(x0, x1);
          pr[r / 2] = *reinterpret_cast<const uint32_t*>(&a);
        }
        if (__any_sync(0xffffffffu, vv == 0.0f)) {  // an entry without values has a weight only
#pragma unroll
          for (int r = 0; r < 8; ++r) pr[r] = vv == 0.0f ? 0u : pr[r];
        }
        // (its place among the columns: see V)
        const int p_row = (t & ~15) + 4 * ((t >> 1) & 3) + 2 * ((t >> 3) & 1) + (t & 1);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<uint4*>(sm + C::kOffP + p_row * 64 + (((2 * half + c) ^ ((p_row >> 1) & 3)) << 4)) = make_uint4(pr[4 * c], pr[4 * c + 1], pr[4 * c + 2], pr[4 * c + 3]);
        fence_proxy_async_smem();
        wait_st();
        fence_before();
        arrive(p_put);
      }
      cp_async_wait_all();
      // ---- the segment's maxima, sums and O^T for the joining kernel
      if (ok && !all_wait(o_full, (done + count - 1) & 1)) ok = false;
      fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a[4];
        l[2 * c].get(a[0], a[1]);
        l[2 * c + 1].get(a[2], a[3]);
        put(c, a[0], a[1], a[2], a[3]);
      }
      // (the ring is free: every tile's codes have been through a product; channels of other words a few banks on)
      float* O = reinterpret_cast<float*>(sm + C::kOffRing);
      constexpr int kOn = D == 128 ? 2 : 4;
      if (ok && w < D / 32) {
        const int e = lane >> 3, ch = (32 + kOn) * word_j(lane & 7) + 8 * e + word_g(lane & 7);
        const float f = e & 1 ? 0.0625f : 1.0f;  // (those channels' codes are x 16)
        uint32_t o[16];
        tmem_ld16(tmem + lanes + C::kColO + 16 * half, o);
        wait_ld();
#pragma unroll
        for (int r = 0; r < 16; ++r) O[(16 * half + r) * C::kPitch + ch] = __uint_as_float(o[r]) * f;
      }
      work_sync();
      if (ok) {
        float* dst = j0 > 0 ? sp.more + (int64_t)blockIdx.x * kMaxRows * (D + kPartHead) : sp.first + q_row * (D + kPartHead);
        float sum = 0.0f;
#pragma unroll 4
        for (int k = 0; k < 16; ++k) sum += get(k);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (eighth == 0 && row < nrow) *reinterpret_cast<float2*>(dst + row * (D + kPartHead) + 4) = make_float2(row_m[row], sum);
#pragma unroll 2
        for (int k = tid; k < nrow * (D / 4); k += kWork) {
          const int r = k / (D / 4), c = 4 * (k % (D / 4));
          const float* from = O + r * C::kPitch + c + kOn * (c / 32);
          const float2 a = *reinterpret_cast<const float2*>(from), b = *reinterpret_cast<const float2*>(from + 2);
          *reinterpret_cast<float4*>(dst + r * (D + kPartHead) + kPartHead + c) = make_float4(a.x, a.y, b.x, b.y);
        }
      }
      fence_before();
    }
    if (!ok) failed = 1;
    __syncthreads();
    fence_after();
    done += count;
    if (failed) break;
  }
  if (failed && tid == 0) set_status(p.status, FT_DEV_TIMEOUT);
  if (warp == kWork / 32) {
    // tensor memory is freed only when nothing issued here is in flight
    const uint32_t lead = lane == 0 ? 1u : 0u;
    if (failed) {
      __shared__ __align__(8) uint64_t drained;
      if (lane == 0) {
        mbar_init(smem_u32(&drained), 1);
        mbar_fence_init();
      }
      __syncwarp();
      commit(smem_u32(&drained), lead);
      all_wait(smem_u32(&drained), 0);
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kCols));
  }
}

template <int D>
static cudaError_t launch(const AttnPagedParams& p, void* workspace, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(tree_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    allowed[dev] = 1;
  }
  Split sp = split_of(workspace, p.B, (int64_t)p.total_q * p.L.nkv * p.G, D, kPerSm * num_sms(), kMaxRows);
  sp.seg = kSegUnits;
  sp.odd = 0.0625f, sp.up = kOUp;
  cudaError_t e = launch_prepare<D>(p, sp, st);
  if (e != cudaSuccess) return e;
  e = launch_served(tree_few_kernel<D>, dim3((unsigned)sp.ctas), dim3(kThreads), Cfg<D>::kSmem, st, 1, p, sp);
  return e != cudaSuccess ? e : launch_join<D>(p, sp, st);
}

}  // namespace few

}  // namespace tree

size_t attn_tree_few_ws(int nkv, int G, int head_dim, int B, int total_q) {
  return tree::split_bytes(B, (int64_t)total_q * nkv * G, head_dim, tree::few::kPerSm * tree::num_sms(), tree::few::kMaxRows);
}

cudaError_t launch_attn_tree_few(const AttnPagedParams& p, int head_dim, void* workspace, cudaStream_t st) {
  return head_dim == 128 ? tree::few::launch<128>(p, workspace, st) : tree::few::launch<64>(p, workspace, st);
}

}  // namespace ft
