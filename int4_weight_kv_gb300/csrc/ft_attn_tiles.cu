// Attention over the paged 4-bit cache for requests with many rows (prompts and chunks
// of prompts), on the fifth-generation tensor cores.
//
// A CTA owns up to 256 rows (tokens x heads of a group, two tiles of M = 128) of one
// request and KV head and walks the visible positions in tiles of 128:
//   S = Q K^T   A = Q from shared memory, B = K codes from shared memory
//   O += P V    A = P from tensor memory (over S's columns), B = V codes from shared memory
// both with FP16 operands and FP32 accumulators in tensor memory (S 2 x 128 columns, O
// 2 x d columns).  K and V are decoded once per CTA for both tiles: codes become FP16
// subnormals (7 integer instructions per 8 values, no offset), in the 128-byte-swizzled
// K-major layout; the order of the channels inside a K step is the cache's own, and Q is
// written in the same order.  The scales stay out of the operands: score = S ks + log2 vs
// in one FMA, the sum of weights takes p / vs (ft_attn_paged.cu).
//
// Roles: two warpgroups of softmax (one row per thread, a tile each), one warpgroup
// decoding (the next tile's bytes in flight in registers), one issuing thread.  While one
// tile's softmax runs, the tensor core works for the other:
//   PV0(j) QK0(j+1) PV1(j) QK1(j+1) ...
// The running max moves only when a score passes it by 2^4, so O is rarely rescaled.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
#include <algorithm>

#include "ft_attn_paged.cuh"

namespace ft {

namespace tiles {

constexpr int kThreads = 512, kRows = 256, kKeys = 128;
constexpr int kMmaWarp = 12;
constexpr int kScaleRing = 4;
// Registers of a thread by role (softmax twice, decode, issue): the sum over the four
// warpgroups is what the block is launched with, kThreads x 128.
constexpr int kRegSoftmax = 192, kRegDecode = 88, kRegIssue = 40;
static_assert(2 * kRegSoftmax + kRegDecode + kRegIssue <= 4 * 128, "more registers than the block has");

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;                 // 128-byte-wide panels of Q and K rows
  static constexpr int kQ = 128 * D * 2;                 // one tile's query operand
  static constexpr int kK = kKeys * D * 2, kV = kKeys * D * 2;  // one stage
  static constexpr int kOffQ = 0, kOffK = 2 * kQ, kOffV = kOffK + 2 * kK, kOffScale = kOffV + 2 * kV;
  static constexpr int kOffBar = kOffScale + kScaleRing * 3 * kKeys * 4;
  static constexpr int kSmem = kOffBar + 256 + 1024;  // 1024: alignment slack
  static constexpr int kColO = 256;                    // tensor memory: S0, S1, then O0, O1
};

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* d) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]), "=r"(d[8]),
        "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15]), "=r"(d[16]),
        "=r"(d[17]), "=r"(d[18]), "=r"(d[19]), "=r"(d[20]), "=r"(d[21]), "=r"(d[22]), "=r"(d[23]), "=r"(d[24]),
        "=r"(d[25]), "=r"(d[26]), "=r"(d[27]), "=r"(d[28]), "=r"(d[29]), "=r"(d[30]), "=r"(d[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// FP32 accumulator, FP16 operands, both K-major.
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major tile of 128-byte-swizzled rows: 8-row atoms of 1024 bytes.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A wait of a whole warp with one outcome: its accesses to tensor memory are warp-wide.
__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Walsh-Hadamard transform of a whole row held by one thread (pairs of channels).
template <int D>
__device__ __forceinline__ void row_fwht(f32x2 (&v)[D / 2], int hb) {
  const f32x2 minus(-1.0f, -1.0f);
  if (hb > 1) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) {
      float a, b;
      v[i].get(a, b);
      v[i] = f32x2(a + b, a - b);
    }
  }
#pragma unroll
  for (int s = 1; s < D / 2; s <<= 1) {
    if (2 * s >= hb) break;
#pragma unroll
    for (int i = 0; i < D / 2; ++i) {
      if (i & s) continue;
      const f32x2 a = v[i], b = v[i + s];
      v[i] = add2(a, b);
      v[i + s] = fma2(b, minus, a);
    }
  }
}

}  // namespace tiles

using namespace tiles;

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnPagedParams p) {
  using C = Cfg<D>;
  constexpr int NJ = D / 32;
  extern __shared__ uint8_t tiles_smem[];
  const uint32_t raw = smem_u32(tiles_smem);
  uint8_t* sm = tiles_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ int find[3];       // request, first row of the CTA's rows (-1: no work), and the blocks of all requests
  __shared__ int warp_tot[16];
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- which rows: block i of all requests' 256-row blocks, the last ones (which see most) first
  const int h = blockIdx.x % p.L.nkv, want = blockIdx.x / p.L.nkv;
  {
    auto blocks = [&](int b, int32_t* status) {
      int row0, n, kv;
      if (!attn_request(p, b, status, row0, n, kv)) return 0;
      return (int)(((int64_t)n * p.G + kRows - 1) / kRows);
    };
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += blocks(b, blockIdx.x == 0 ? p.status : nullptr);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_tot[warp] = inc;
    if (tid == 0) find[1] = -1;
    __syncthreads();
    int at = inc - sum, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += warp_tot[w];
      total += warp_tot[w];
    }
    const int i = total - 1 - want;
    if (i >= at && i < at + sum) {
      for (int b = b0; b < b1; ++b) {
        const int nb = blocks(b, nullptr);
        if (i < at + nb) {
          find[0] = b;
          find[1] = (i - at) * kRows;
          break;
        }
        at += nb;
      }
    }
    __syncthreads();
  }
  const int b = find[0], r0 = find[1];
  if (r0 < 0) return;
  const int row0 = p.cu[b], n = p.cu[b + 1] - row0;
  int kv = p.kv_len[b];
  if (kv < 0 || ((kv + (int64_t)p.L.psize - 1) >> p.L.pshift) > p.table_stride) kv = 0;
  const int nrow = min((int)((int64_t)n * p.G - r0), kRows);  // rows of this CTA
  const int ntile = nrow > 128 ? 2 : 1;
  const int last = kv - n + (r0 + nrow - 1) / p.G;               // last visible position of any row
  const int nkt = last >= 0 ? last / kKeys + 1 : 0;
  const int* table = p.table + (size_t)b * p.table_stride;

  const uint32_t bar = sm32 + C::kOffBar;
  const uint32_t q_full = bar, s_full = bar + 16, p_full = bar + 32, o_full = bar + 48, k_full = bar + 64,
                 k_empty = bar + 80, v_full = bar + 96, v_empty = bar + 112, sc_full = bar + 128, drained = bar + 160;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 128);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(k_full + 8 * i, 128);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 128);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full + 8 * i, 128);
    mbar_init(drained, 1);
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
  float* scales = reinterpret_cast<float*>(sm + C::kOffScale);  // [ring][ks, lv, rs][kKeys]
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax: one row per thread
    regs_up<kRegSoftmax>();
    const int t = warp >> 2, row = tid & 127, r = r0 + 128 * t + row;
    const bool live = 128 * t + row < nrow;
    const int tok = min(r / p.G, n - 1), hh = r - (r / p.G) * p.G;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    if (t < ntile) {
      {  // the rotated query row as the FP16 operand, channels in the order of the cache's words
        f32x2 v[D / 2];
        const uint16_t* src = p.q + (row0 + tok) * p.q_stride + (int64_t)(h * p.G + hh) * D;
        if (!live) {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) v[i] = f32x2(0.0f, 0.0f);
        } else if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = f32x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) v[i] = f32x2(bf16_bits_to_f32(__ldg(src + 2 * i)), bf16_bits_to_f32(__ldg(src + 2 * i + 1)));
        }
        row_fwht<D>(v, p.hb);
        const float f0 = p.qscale * p.norm, f1 = f0 * 0.0625f;
        bool bad = false;
        uint8_t* qs = sm + C::kOffQ + t * C::kQ + row * 128;
#pragma unroll
        for (int w = 0; w < D / 8; ++w) {  // word w = (tig, j): channels 32 j + 2 tig + 8 e + {0, 1}
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, c;
            v[16 * (w % NJ) + (w / NJ) + 4 * e].get(a, c);
            a *= (e & 1) ? f1 : f0;
            c *= (e & 1) ? f1 : f0;
            const float top = (e & 1) ? 4094.0f : 65504.0f;
            bad |= !(fabsf(a) <= top) || !(fabsf(c) <= top);
            const __half2 hv = __floats2half2_rn(a, c);
            o[e] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          *reinterpret_cast<uint4*>(qs + (w / 8) * (128 * 128) + (((w % 8) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (bad) set_status(p.status, FT_DEV_RANGE);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full + 8 * t);

      const int lim = kv - n + tok;  // last position this row sees
      const int lim_all = kv - n + (r0 + 128 * t + 32 * (warp & 3)) / p.G;  // and that every row of the warp sees
      float m = -INFINITY;
      f32x2 l2(0.0f, 0.0f);
      for (int j = 0; j < nkt; ++j) {
        const float* sc = scales + (j % kScaleRing) * 3 * kKeys;
        if (!all_wait(s_full + 8 * t, j & 1) || !all_wait(sc_full + 8 * (j % kScaleRing), (j / kScaleRing) & 1)) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(tmem + lane_base + 128 * t + c, s + c);
        wait_ld();
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kKeys; c += 4) {
          const float4 ks = *reinterpret_cast<const float4*>(sc + c), lv = *reinterpret_cast<const float4*>(sc + kKeys + c);
          float x0, x1, x2, x3;
          fma2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), f32x2(ks.x, ks.y), f32x2(lv.x, lv.y)).get(x0, x1);
          fma2(f32x2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), f32x2(ks.z, ks.w), f32x2(lv.z, lv.w)).get(x2, x3);
          s[c] = __float_as_uint(x0), s[c + 1] = __float_as_uint(x1), s[c + 2] = __float_as_uint(x2), s[c + 3] = __float_as_uint(x3);
        }
        if (kKeys * j + kKeys - 1 > lim_all) {  // a tile that some row of the warp sees in part
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] = kKeys * j + c <= lim ? s[c] : 0xFF800000u;
        }
#pragma unroll
        for (int c = 0; c < kKeys; ++c) mx = fmaxf(mx, __uint_as_float(s[c]));
        const bool need = mx > m + kPLazy;
        if (__any_sync(0xffffffffu, need)) {
          const float to = need ? mx : m;
          const float f = to == m ? 1.0f : ex2(m - to);
          m = to;
          if (j > 0) {
            l2 = mul2(l2, f32x2(f, f));
            if (!all_wait(o_full + 8 * t, (j - 1) & 1)) {  // the tensor core is done with O
              ok = false;
              break;
            }
            fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(tmem + lane_base + C::kColO + D * t + c, o);
            }
          }
        }
        const float u = kPBias - (m == -INFINITY ? 0.0f : m);
        const f32x2 u2(u, u);
#pragma unroll
        for (int c0 = 0; c0 < kKeys; c0 += 64) {
          uint32_t o[32];
#pragma unroll
          for (int c = c0; c < c0 + 64; c += 4) {
            const float4 rs = *reinterpret_cast<const float4*>(sc + 2 * kKeys + c);
            float x0, x1, x2, x3;
            add2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), u2).get(x0, x1);
            add2(f32x2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), u2).get(x2, x3);
            x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
            l2 = fma2(f32x2(x0, x1), f32x2(rs.x, rs.y), l2);
            l2 = fma2(f32x2(x2, x3), f32x2(rs.z, rs.w), l2);
            const __half2 h0 = __floats2half2_rn(x0, x1), h1 = __floats2half2_rn(x2, x3);
            o[(c - c0) / 2] = *reinterpret_cast<const uint32_t*>(&h0);
            o[(c - c0) / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          }
          tmem_st32(tmem + lane_base + 128 * t + c0 / 2, o);
        }
        wait_st();
        fence_before();
        mbar_arrive(p_full + 8 * t);
      }
      // ---- epilogue: O / l, the rotation undone, BF16
      if (ok && nkt > 0 && !all_wait(o_full + 8 * t, (nkt - 1) & 1)) ok = false;
      if (ok) {
        fence_after();
        float la, lb;
        l2.get(la, lb);
        const float l = la + lb, inv = l == 0.0f ? 0.0f : kOUp / l;  // a row that sees nothing: zeros
        const f32x2 f0(inv, inv), f1(inv * 0.0625f, inv * 0.0625f);
        f32x2 v[D / 2];
        if (nkt > 0) {
          uint32_t o[D];
#pragma unroll
          for (int c = 0; c < D; c += 32) tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o + c);
          wait_ld();
#pragma unroll
          for (int i = 0; i < D / 2; ++i)
            v[i] = mul2(f32x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), (i & 4) ? f1 : f0);
        } else {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) v[i] = f32x2(0.0f, 0.0f);
        }
        row_fwht<D>(v, p.hb);
        const f32x2 norm2(p.norm, p.norm);
        if (live) {
          uint16_t* dst = p.o + (row0 + tok) * p.o_stride + (int64_t)(h * p.G + hh) * D;
          const bool aligned = (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a, c;
              mul2(v[4 * i + k], norm2).get(a, c);
              const __nv_bfloat162 bv = __floats2bfloat162_rn(a, c);
              w[k] = *reinterpret_cast<const uint32_t*>(&bv);
            }
            if (aligned) {
              reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                dst[8 * i + 2 * k] = (uint16_t)w[k];
                dst[8 * i + 2 * k + 1] = (uint16_t)(w[k] >> 16);
              }
            }
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ decode K and V
    regs_down<kRegDecode>();
    const int w4 = warp - 8, dt = tid - 256;
    constexpr int KR = D / 32;  // K: 16-byte (d = 128) or 8-byte pieces, four (tig) a key
    // round i covers keys 32 i + 8 w4 .. + 7 of a tile: this lane's K piece is (key lane & 7, column lane >> 3),
    // its V words are those of channels (g = lane & 7, j = lane >> 3), for d = 64 (j = (lane >> 3) & 1)
    // with the pairs split between the lane halves
    uint32_t kw[4][KR];
    uint32_t vw[4][D == 128 ? 4 : 2];
    uint32_t sc_next = 0;
    bool sc_ok = false;
    auto page_of = [&](int pos) {  // -1 behind the end; a page outside the pool is flagged
      if (pos >= kv) return -1;
      const int page = __ldg(table + (pos >> p.L.pshift));
      if (page >= 0 && page < p.L.npages) return page;
      set_status(p.status, FT_DEV_RANGE);
      return -1;
    };
    auto load_k = [&](int j) {
      const int pos = kKeys * j + dt;  // this thread's scale
      const int sp = page_of(pos);
      sc_ok = sp >= 0;
      if (sc_ok)
        sc_next = ld_stream_u32(p.pages + paged_block(p.L, sp, h) + p.L.soff + 4 * (pos & (p.L.psize - 1)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p0 = kKeys * j + 32 * i + 8 * w4, page = page_of(p0);
#pragma unroll
        for (int k = 0; k < KR; ++k) kw[i][k] = 0u;
        if (page >= 0) {
          const uint8_t* src = p.pages + paged_block(p.L, page, h) + ((p0 & (p.L.psize - 1)) + (lane & 7)) * (D / 2) + (lane >> 3) * (D / 8);
          if constexpr (D == 128) {
            const uint4 q = ld_stream_v4(src);
            kw[i][0] = q.x, kw[i][1] = q.y, kw[i][2] = q.z, kw[i][3] = q.w;
          } else {
            const uint2 q = ld_stream_v2(src);
            kw[i][0] = q.x, kw[i][1] = q.y;
          }
        }
      }
    };
    auto load_v = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p0 = kKeys * j + 32 * i + 8 * w4, page = page_of(p0);
        constexpr int NW = D == 128 ? 4 : 2;
#pragma unroll
        for (int k = 0; k < NW; ++k) vw[i][k] = 0u;
        if (page >= 0) {
          const uint8_t* blk = p.pages + paged_block(p.L, page, h) + p.L.voff;
          const int pair0 = (p0 & (p.L.psize - 1)) >> 1, g = lane & 7;
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const int pair = D == 128 ? pair0 + k : pair0 + 2 * (lane >> 4) + k, jj = D == 128 ? lane >> 3 : (lane >> 3) & 1;
            vw[i][k] = ld_stream_u32(blk + pair * D + (g ^ paged_v_turn<D>(pair)) * (D / 8) + 4 * jj);
          }
        }
      }
    };
    if (nkt > 0) {
      load_k(0);
      load_v(0);
    }
    for (int j = 0; j < nkt; ++j) {
      const int st = j & 1;
      if (j >= 2 && !mbar_wait(k_empty + 8 * st, ((j - 2) >> 1) & 1)) {
        ok = false;
        break;
      }
      {
        uint8_t* kd = sm + C::kOffK + st * C::kK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * i + 8 * w4 + (lane & 7);
#pragma unroll
          for (int k = 0; k < KR; ++k) {
            const int w = (lane >> 3) * NJ + k;  // word of the entry: slots 8 w .. 8 w + 7 of the operand's row
            uint32_t r[4];
            paged_word(kw[i][k], r);
            *reinterpret_cast<uint4*>(kd + (w / 8) * (kKeys * 128) + key * 128 + (((w % 8) ^ (key & 7)) << 4)) =
                make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
        // scales of the tile; positions behind the end (or on no page) are masked by them
        float* sc = scales + (j % kScaleRing) * 3 * kKeys;
        const float vs = fmaxf(__uint_as_float(sc_next & 0xFFFF0000u), kMinScale);
        sc[dt] = sc_ok ? __uint_as_float(sc_next << 16) * kKsUp : 0.0f;
        sc[kKeys + dt] = sc_ok ? lg2(vs) : -INFINITY;
        sc[2 * kKeys + dt] = sc_ok ? rcp(vs) : 0.0f;
      }
      fence_proxy_async_smem();
      mbar_arrive(sc_full + 8 * (j % kScaleRing));
      mbar_arrive(k_full + 8 * st);
      if (j + 1 < nkt) load_k(j + 1);
      if (j >= 2 && !mbar_wait(v_empty + 8 * st, ((j - 2) >> 1) & 1)) {
        ok = false;
        break;
      }
      {
        uint8_t* vd = sm + C::kOffV + st * C::kV;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int chunk = 4 * i + w4;  // 8 positions
          uint8_t* panel = vd + (chunk / 8) * (D * 128);
          if constexpr (D == 128) {
            uint32_t r[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) paged_word(vw[i][k], r[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ch = 32 * (lane >> 3) + (lane & 7) + 8 * e;
              *reinterpret_cast<uint4*>(panel + ch * 128 + (((chunk % 8) ^ (ch & 7)) << 4)) =
                  make_uint4(r[0][e], r[1][e], r[2][e], r[3][e]);
            }
          } else {
            uint32_t r[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) paged_word(vw[i][k], r[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ch = 32 * ((lane >> 3) & 1) + (lane & 7) + 8 * e;
              *reinterpret_cast<uint2*>(panel + ch * 128 + (((chunk % 8) ^ (ch & 7)) << 4) + 8 * (lane >> 4)) =
                  make_uint2(r[0][e], r[1][e]);
            }
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(v_full + 8 * st);
      if (j + 1 < nkt) load_v(j + 1);
    }
  } else {
    regs_down<kRegIssue>();
    if (warp == kMmaWarp && lane == 0) {
      // ---------------------------------------------------------- tensor-core issue
      constexpr uint32_t id_qk = idesc_f16(128, kKeys), id_pv = idesc_f16(128, D);
      auto qk = [&](int t, int j) {
        const uint32_t qa = sm32 + C::kOffQ + t * C::kQ, ka = sm32 + C::kOffK + (j & 1) * C::kK;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (ks / 4) * (128 * 128) + 32 * (ks % 4);
          mma_ss(tmem + 128 * t, desc_sw128(qa + o), desc_sw128(ka + o), id_qk, ks > 0 ? 1u : 0u);
        }
        commit(s_full + 8 * t);
      };
      auto pv = [&](int t, int j) {
        const uint32_t va = sm32 + C::kOffV + (j & 1) * C::kV;
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_ts(tmem + C::kColO + D * t, tmem + 128 * t + 8 * ks, desc_sw128(va + (ks / 4) * (D * 128) + 32 * (ks % 4)), id_pv,
                 j > 0 || ks > 0 ? 1u : 0u);
        commit(o_full + 8 * t);
      };
      if (nkt > 0) {
        ok = mbar_wait(k_full, 0);
        for (int t = 0; ok && t < ntile; ++t) {
          ok = mbar_wait(q_full + 8 * t, 0);
          fence_after();
          if (ok) qk(t, 0);
        }
        if (ok) commit(k_empty);
      }
      for (int j = 0; ok && j < nkt; ++j) {
        const bool more = j + 1 < nkt;
        for (int t = 0; ok && t < ntile; ++t) {
          ok = (t > 0 || mbar_wait(v_full + 8 * (j & 1), (j >> 1) & 1)) && mbar_wait(p_full + 8 * t, j & 1);
          if (!ok) break;
          fence_after();
          pv(t, j);
          if (t == ntile - 1) commit(v_empty + 8 * (j & 1));
          if (more) {
            if (t == 0) ok = mbar_wait(k_full + 8 * ((j + 1) & 1), ((j + 1) >> 1) & 1);
            if (!ok) break;
            fence_after();
            qk(t, j + 1);
            if (t == ntile - 1) commit(k_empty + 8 * ((j + 1) & 1));
          }
        }
      }
      // tensor memory is freed only when nothing issued here is in flight
      commit(drained);
      if (!mbar_wait(drained, 0)) ok = false;
    }
    __syncwarp();
  }
  if (!ok) set_status(p.status, FT_DEV_TIMEOUT);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

template <int D>
static cudaError_t launch_tiles_d(const AttnPagedParams& p, cudaStream_t st) {
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
    if (fa.numRegs * 4 < 2 * kRegSoftmax + kRegDecode + kRegIssue) return cudaErrorInvalidConfiguration;
    allowed[dev] = 1;
  }
  // an upper bound of the 256-row blocks of all requests
  const int64_t blocks = ((int64_t)p.total_q * p.G) / kRows + std::min(p.B, p.total_q);
  if (blocks * p.L.nkv > INT32_MAX) return cudaErrorInvalidConfiguration;
  attn_tiles_kernel<D><<<(unsigned)(blocks * p.L.nkv), kThreads, Cfg<D>::kSmem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_attn_tiles(const AttnPagedParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch_tiles_d<128>(p, st) : launch_tiles_d<64>(p, st);
}

}  // namespace ft
