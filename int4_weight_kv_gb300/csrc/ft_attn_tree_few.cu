// Attention of small draft trees (up to 32 rows, tokens x heads of a group) over the paged 4-bit cache, on the
// fifth-generation tensor cores with the positions as the products' rows:
//   S^T = K Q^T     A = K codes from tensor memory (128 positions), B = the query rows from shared memory (N = 32)
//   O^T += V^T P^T  A = V codes from tensor memory (the channels), B = P from shared memory
// so that a thread has one position's scores of all rows: the position's scales are two of its registers, the codes need
// no scale, and as an FP16 subnormal each costs 7 instructions for eight of them.  What a row of products with 128 of them
// would do for rows that are not there is left out, and shared memory holds 16 KB of operands where it held 160.
// How the work is shared out and joined: ft_attn_tree.cuh; the arithmetic: that of the kernel for few rows in
// ft_attn_paged.cu.
//
// A CTA has four warps that work (a position each for K and the softmax, a channel each for V) and one that issues; two
// CTAs an SM, whose phases fill each other's waits:
//   tile i: K decoded (while P V of tile i - 1 runs), V decoded (while Q K^T runs), softmax
// Bytes come by 16-byte asynchronous copies, a tile ahead.  The running max moves when a score passes it by 2^4.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
#include "ft_attn_tree.cuh"

namespace ft {

namespace tree {

namespace few {

constexpr int kThreads = 160, kWork = 128, kMaxRows = 32, kPerSm = 2;
constexpr int kSegUnits = 3;  // a segment's cost beside its positions, in tiles of them

template <int D>
struct Cfg {
  static constexpr int kStage = kKeys * D;  // K and V of a tile, as they are
  static constexpr int kOffQ = 0, kOffP = kMaxRows * D * 2, kOffRing = kOffP + kKeys * kMaxRows * 2, kOffRows = kOffRing + 2 * kStage;
  static constexpr int kOffBar = kOffRows + kMaxRows * 8 + 4 * kMaxRows * 4 + 3 * kMaxRows * 4;
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
// Whether any of the working threads says so.
__device__ __forceinline__ bool any_of_work(bool x) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 1, 128, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"((uint32_t)x)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ void work_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) tree_few_kernel(const AttnPagedParams p, const Split sp) {
  using C = Cfg<D>;
  constexpr int CE = D / 32;  // 16-byte chunks of a K entry
  extern __shared__ uint8_t few_tree_smem[];
  const uint32_t raw = smem_u32(few_tree_smem);
  uint8_t* sm = few_tree_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ int4 seg[3];
  __shared__ int failed;
  __shared__ uint32_t tmem_slot;
  float** row_at = reinterpret_cast<float**>(sm + C::kOffRows);                        // [32] where a row's partial goes
  float* sums = reinterpret_cast<float*>(sm + C::kOffRows + kMaxRows * 8);             // [4][32]
  float *row_m = sums + 4 * kMaxRows, *row_u = row_m + kMaxRows;                       // running max, kPBias - max (kPBias for none yet)
  uint32_t* row_mask = reinterpret_cast<uint32_t*>(row_u + kMaxRows);                  // which new tokens a row sees
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  const uint32_t bar = sm32 + C::kOffBar, k_put = bar, s_full = bar + 8, p_put = bar + 16, o_full = bar + 24;
  if (tid == 0) {
    mbar_init(k_put, 4);  // (a lane of each working warp)
    mbar_init(p_put, 4);
    mbar_init(s_full, 1);
    mbar_init(o_full, 1);
    mbar_fence_init();
    failed = 0;
  }
  if (warp == 4) {
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

  // ---- this CTA's share
  const int64_t units = __ldcg(sp.pref + p.B);
  const int shares = shares_of(units, gridDim.x), cta = min((int)blockIdx.x, shares);
  const int64_t u = share_begin(units, shares, cta);
  int64_t off = 0, left = share_begin(units, shares, min(cta + 1, shares)) - u;  // place in the request's units, units left
  int b = -1, row0 = 0, n = 0, kv = 0;
  bool fresh_b = true;
  if (warp == 4 && left > 0) {
    // the last request whose prefix sum is <= u, by up to three steps of 32 candidates
    b = 0;
    for (int st = p.B > 1024 ? 1024 : p.B > 32 ? 32 : 1; st; st >>= 5) {
      const int i = b + (lane + 1) * st;
      b += st * __popc(__ballot_sync(0xffffffffu, i < p.B && __ldcg(sp.pref + min(i, p.B)) <= u));
    }
    off = u - __ldcg(sp.pref + b);
  }
  uint32_t done = 0;  // tiles of the segments before this one
  while (true) {
    if (warp == 4) {  // the next segment: positions j0 .. j1 - 1 (tiles) of request b for head h
      int j0 = 0, j1 = 0, h = 0;
      bool found = false;
      while (b >= 0 && b < p.B && left > 0 && !found) {
        if (fresh_b) {
          if (!attn_request(p, b, nullptr, row0, n, kv)) n = 0;
          fresh_b = false;
        }
        const Units x(p, n, kv, sp.seg);
        if (n == 0 || off >= x.total) {
          ++b, off = 0, fresh_b = true;
          continue;
        }
        h = (int)(off / x.last);
        const int64_t at = off - h * x.last, go = min(left, x.last - at);
        j0 = x.tile(0, at), j1 = x.tile(0, at + go);
        off += go, left -= go;
        found = j0 < j1;  // (else the share ends in what the segment costs beside its positions)
      }
      if (lane == 0) {
        seg[0] = make_int4(found ? b : -1, row0, n, kv);
        seg[1] = make_int4(h, j0, j1, 0);
      }
    }
    __syncthreads();
    const int4 s0 = seg[0], s1 = seg[1];
    if (s0.x < 0) break;
    const int s_b = s0.x, s_row0 = s0.y, s_n = s0.z, s_kv = s0.w, h = s1.x, j0 = s1.y, count = s1.z - s1.y;
    const int nrow = s_n * p.G;
    if (warp == 4) {
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
    } else {
      // ------------------------------------------------------------ work
      const uint32_t lanes = (uint32_t)(32 * warp) << 16;
      const int* table = p.table + (int64_t)s_b * p.table_stride;
      const int fresh = s_kv - s_n;  // positions before this one are seen by every row
      const uint64_t page_bytes = (uint64_t)((uint32_t)p.L.nkv * p.L.block);
      const uint8_t* base = p.pages + (size_t)h * p.L.block;
      // query rows (zeros behind the last), where the rows' partials go, and their masks
      for (int i = tid; i < kMaxRows * (D / 8); i += kWork) {
        const int r = i / (D / 8), c = i % (D / 8), rr = min(r, nrow - 1), tok = rr / p.G;
        const uint16_t* src = sp.q + ((int64_t)(s_row0 + tok) * (p.L.nkv * p.G) + h * p.G + (rr - tok * p.G)) * D + 8 * c;
        cp_async16_zfill(sm32 + C::kOffQ + chunk_at(kMaxRows, r, c), src, r < nrow);
      }
      if (tid < kMaxRows) {
        const int rr = min(tid, nrow - 1), tok = rr / p.G;
        row_at[tid] = (j0 > 0 ? sp.more + ((int64_t)blockIdx.x * sp.rows + rr) * (D + kPartHead)
                              : sp.first + ((int64_t)(s_row0 + tok) * (p.L.nkv * p.G) + h * p.G + (rr - tok * p.G)) * (D + kPartHead));
        row_mask[tid] = tid < nrow ? p.mask[(int64_t)(s_row0 + tok) * p.mask_stride] : 0u;  // (up to 32 new tokens: one word)
        row_m[tid] = -INFINITY;
      }
      // The bytes of tile i: K entry by entry (chunks turned so that 8 lanes' reads meet 8 banks), V as it is; pages outside
      // the pool and behind the end are page 0 (no scale, and hidden).  Pages are looked up a tile further ahead.
      int pages[CE], own_page;
      auto look_up = [&](int i) {
        const int p0 = kKeys * (j0 + i);
        auto at = [&](int pos) { return i < count && pos < s_kv ? __ldg(table + (pos >> p.L.pshift)) : -1; };
#pragma unroll
        for (int k = 0; k < CE; ++k) pages[k] = at(p0 + (tid + kWork * k) / (16 * CE) * 16);
        own_page = at(p0 + tid);
      };
      uint32_t sc_next = 0u;
      bool there_next = false;
      auto copy = [&](int i) {
        const uint32_t st = sm32 + C::kOffRing + (i & 1) * C::kStage;
        const int p0 = kKeys * (j0 + i);
#pragma unroll
        for (int k = 0; k < CE; ++k) {
          const int q = tid + kWork * k, entry = q / CE, c = q % CE, pair = q / (2 * CE), c2 = q % (2 * CE);
          const uint8_t* pg = base + ((uint32_t)pages[k] < (uint32_t)p.L.npages ? (uint32_t)pages[k] : 0u) * page_bytes;
          const uint32_t turn = D == 128 ? c ^ ((entry >> 1) & 3) : c;
          cp_async16(st + entry * (D / 2) + 16 * turn, pg + ((p0 + entry) & (p.L.psize - 1)) * (D / 2) + 16 * c);
          cp_async16(st + kKeys * D / 2 + pair * D + 16 * c2, pg + p.L.voff + ((p0 + 2 * pair) & (p.L.psize - 1)) * (D / 2) + 16 * c2);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const int pos = p0 + tid;
        there_next = i < count && pos < s_kv && (uint32_t)own_page < (uint32_t)p.L.npages;
        if (i < count && pos < s_kv && !there_next) set_status(p.status, FT_DEV_RANGE);
        sc_next = ld_stream_u32(base + (there_next ? (uint32_t)own_page : 0u) * page_bytes + p.L.soff + 4 * (pos & (p.L.psize - 1)));
      };
      look_up(0);
      copy(0);
      look_up(1);
      float l[kMaxRows];
#pragma unroll
      for (int r = 0; r < kMaxRows; ++r) l[r] = 0.0f;
      int i = 0;
      for (; i < count; ++i) {
        const uint32_t parity = (done + i) & 1;
        const uint32_t sc = sc_next;
        const bool there = there_next;
        // (behind the last tile: a copy of no use, as the loads' ends are waited for by number)
        work_sync();  // the other stage's bytes have been read by all
        copy(i + 1);
        look_up(i + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        work_sync();
        const uint8_t* st = sm + C::kOffRing + (i & 1) * C::kStage;
        // ---- K: this thread's position (the operand's room is free: S of tile i - 1 was waited for)
        fence_after();
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint32_t x[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int ch = 2 * hf + c;
            const uint4 q = *reinterpret_cast<const uint4*>(st + tid * (D / 2) + 16 * (D == 128 ? ch ^ ((tid >> 1) & 3) : ch));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t r[4];
              paged_word(w[k], r);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[16 * c + 4 * k + e] = r[e];
            }
          }
          tmem_st32(tmem + lanes + C::kColK + 32 * hf, x);
        }
        wait_st();
        if (i == 0) fence_proxy_async_smem();  // (the query rows)
        fence_before();
        arrive(k_put);
        // ---- V: this thread's channel, when P V of tile i - 1 is through with the operands
        if (i > 0 && !all_wait(o_full, (done + i - 1) & 1)) ok = false;
        fence_after();
        if (warp < D / 32) {
          const int g = lane & 7, e = lane >> 3;
          const uint32_t order = (e & 2) ? 0x2301u : 0x3210u, shift = e & 1, keep = (e & 1) ? 0x80708070u : 0x80078007u;
          const uint8_t* v = st + kKeys * D / 2 + 4 * warp;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(v + (32 * hf + k) * D + (g ^ paged_v_turn<D>(k)) * (D / 8));
              x[k] = (prmt(w, 0u, order) << shift) & keep;
            }
            tmem_st32(tmem + lanes + C::kColV + 32 * hf, x);
          }
        }
        // ---- softmax: this thread's position, all rows
        const float ks = __uint_as_float(sc << 16) * kKsUp, vv = __uint_as_float(sc & 0xFFFF0000u);
        const float vs = vv == 0.0f ? kNoScale : fmaxf(vv, kMinScale);
        // (a scale from 2^110 on, kTooLarge, makes this and with it the scores NaN, whatever they were)
        const float lv = fmaf(fmaf(vv, kKsUp, ks), 0.0f, lg2(vs)), rs = there ? rcp(vs) : 0.0f;
        const int at = kKeys * (j0 + i) + tid - fresh;  // the position among the new tokens
        if (!all_wait(s_full, parity)) ok = false;
        fence_after();
        uint32_t sr[kMaxRows];
        tmem_ld32(tmem + lanes + C::kColS, sr);
        wait_ld();
        float s[kMaxRows];
#pragma unroll
        for (int r = 0; r < kMaxRows; ++r) s[r] = fmaf(__uint_as_float(sr[r]), ks, lv);
        if (!__all_sync(0xffffffffu, there && at < 0)) {
#pragma unroll
          for (int r = 0; r < kMaxRows; ++r) {
            const bool seen = there && (at < 0 || ((row_mask[r] >> (at & 31)) & 1u));  // (at < n <= 32 where it is there)
            s[r] = seen ? s[r] : -INFINITY;  // whatever the entry holds
          }
        }
        float over = -INFINITY;
#pragma unroll
        for (int r = 0; r < kMaxRows; r += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(row_m + r);
          over = max3(over, s[r] - m4.x, s[r + 1] - m4.y);
          over = max3(over, s[r + 2] - m4.z, s[r + 3] - m4.w);
        }
        // (-infinity less -infinity is no number, and not the larger: a row without a max yet moves by the first tile's rule)
        if (any_of_work(over > kPLazy || i == 0 || !ok)) {
          if (any_of_work(!ok)) {
            ok = false;
            break;
          }
          float own = -INFINITY;  // lane r: the warp's max of row r
#pragma unroll
          for (int r = 0; r < kMaxRows; ++r) {
            const float x = s[r] == s[r] ? s[r] : -INFINITY;
            const int bits = __float_as_int(x);
            const int top = __reduce_max_sync(0xffffffffu, bits >= 0 ? bits : bits ^ 0x7FFFFFFF);
            if (lane == r) own = __int_as_float(top >= 0 ? top : top ^ 0x7FFFFFFF);
          }
          sums[32 * warp + lane] = own;
          work_sync();
          const float m_old = row_m[lane];
          const float m_new = fmaxf(fmaxf(fmaxf(sums[lane], sums[32 + lane]), fmaxf(sums[64 + lane], sums[96 + lane])), m_old);
          const float fac = m_old == m_new ? 1.0f : ex2(m_old - m_new);
          work_sync();
          if (warp == 0) {
            row_m[lane] = m_new;
            row_u[lane] = kPBias - (m_new == -INFINITY ? 0.0f : m_new);
            sums[lane] = fac;
          }
          work_sync();
          if (i > 0) {
            uint32_t o[kMaxRows];
            tmem_ld32(tmem + lanes + C::kColO, o);
            wait_ld();
#pragma unroll
            for (int r = 0; r < kMaxRows; ++r) {
              const float f = sums[r];
              l[r] *= f;
              o[r] = __float_as_uint(__uint_as_float(o[r]) * f);
            }
            tmem_st32(tmem + lanes + C::kColO, o);
          }
          work_sync();
        }
        uint32_t pr[kMaxRows / 2];
#pragma unroll
        for (int r = 0; r < kMaxRows; r += 4) {
          const float4 u4 = *reinterpret_cast<const float4*>(row_u + r);
          const float x0 = ex2(s[r] + u4.x), x1 = ex2(s[r + 1] + u4.y), x2 = ex2(s[r + 2] + u4.z), x3 = ex2(s[r + 3] + u4.w);
          l[r] = fmaf(x0, rs, l[r]), l[r + 1] = fmaf(x1, rs, l[r + 1]);
          l[r + 2] = fmaf(x2, rs, l[r + 2]), l[r + 3] = fmaf(x3, rs, l[r + 3]);
          const __half2 a = __floats2half2_rn(x0, x1), c = __floats2half2_rn(x2, x3);
          pr[r / 2] = vv == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&a);
          pr[r / 2 + 1] = vv == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&c);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(sm + C::kOffP + tid * 64 + ((c ^ ((tid >> 1) & 3)) << 4)) = make_uint4(pr[4 * c], pr[4 * c + 1], pr[4 * c + 2], pr[4 * c + 3]);
        fence_proxy_async_smem();
        wait_st();
        fence_before();
        arrive(p_put);
      }
      cp_async_wait_all();
      // ---- the segment's maxima, sums and O^T for the joining kernel
      if (ok && !all_wait(o_full, (done + count - 1) & 1)) ok = false;
      fence_after();
      // the rows' sums over the positions: lane r has row r's after five exchanges
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) {
          const bool high = lane & o;
          const float send = high ? l[k] : l[k + o], keep = high ? l[k + o] : l[k];
          l[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      work_sync();
      sums[32 * warp + lane] = l[0];
      work_sync();
      if (ok) {
        if (tid < nrow) *reinterpret_cast<float2*>(row_at[tid] + 4) = make_float2(row_m[tid], sums[tid] + sums[32 + tid] + sums[64 + tid] + sums[96 + tid]);
        if (warp < D / 32) {
          uint32_t o[kMaxRows];
          tmem_ld32(tmem + lanes + C::kColO, o);
          wait_ld();
          const float f = (tid & 8) ? 0.0625f : 1.0f;  // (those channels' codes are x 16)
#pragma unroll
          for (int r = 0; r < kMaxRows; ++r)
            if (r < nrow) row_at[r][kPartHead + tid] = __uint_as_float(o[r]) * f;
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
  if (warp == 4) {
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
