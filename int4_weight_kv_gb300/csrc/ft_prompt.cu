// Causal attention of packed prompts over their own BF16 rows, on the fifth-generation tensor cores.
//
//   o_i = sum_j p_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) q_i . k_j - m),  j <= i
//
// A CTA owns two tiles of up to 128 rows (tokens x heads of a group, so that a KV head's rows are read once
// for all of its query heads) of one sequence and walks the positions that they see in tiles of 128:
//   S = Q K^T   A = Q, B = K from shared memory (both K-major)
//   O += P V    A = P from tensor memory (over S's columns), B = V from shared memory (as it lies there: MN-major)
// with BF16 operands and FP32 accumulators in tensor memory (S 2 x 128 columns, O 2 x d).
//
// Roles: two warpgroups of softmax (one row per thread, a tile each); a warp of which one thread issues the
// TMA copies of Q, K and V; a warp of which one issues the products, for the tiles by turns
//   PV0(j) QK0(j+1) PV1(j) QK1(j+1) ...
// so that the tensor core works for one while the other's softmax runs; and two warps that look through the V
// tiles which some row sees in part: rows behind the sequence's end become zeros, and so do rows that are not
// finite (0 x infinity would reach the rows before them), which are noted for the rows that see them.
// The running max moves only when a score passes it by 2^8 (P is BF16, sums are FP32), so O is rarely rescaled.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
#include <cuda.h>

#include <algorithm>

#include "ft_tc.cuh"

namespace ft {

namespace prompt {

using namespace tiles;

constexpr int kThreads = 384, kKeys = 128;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLookWarp = 11;  // (two issuing warps)
constexpr float kLazy = 8.0f;
constexpr int kPassLeft = 1;  // products of a batch issued behind the end of its turn (1, 2, 3, 5: 344, 349, 360, 371 us for 8192 tokens)
// Registers of a thread: softmax twice, the others; the sum over the three warpgroups is what the block is
// launched with, kThreads x kRegLaunch.
constexpr int kRegSoftmax = 208, kRegOther = 88, kRegLaunch = 168;
static_assert(2 * kRegSoftmax + kRegOther <= 3 * kRegLaunch, "more registers than the block has");

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;              // Q, K or V: 128 rows
  static constexpr int kSlots = D == 128 ? 5 : 8;         // of the ring that K and V tiles come through: K0 V0 K1 V1 ...
  static constexpr int kOffQ = 0, kOffRing = 2 * kTile, kOffBar = kOffRing + kSlots * kTile;
  static constexpr int kSmem = kOffBar + 512 + 1024;      // 1024: alignment slack
  static constexpr int kColO = 256;                       // tensor memory: S0, S1, then O0, O1
};

struct Params {
  const uint16_t* q;
  uint16_t* o;
  int64_t o_stride;
  const int32_t* cu;
  int32_t* status;
  int B, total, max_len, nkv, G, ntile;
  float scale;  // x log2(e)
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// V's operand: 64-channel panels of 128 rows (leading offset), groups of 8 rows (stride, as K-major's).
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr) { return ((saddr & 0x3FFFF) >> 4) | ((uint32_t)(128 * 128) >> 4 << 16); }
constexpr uint32_t kBMn = 1u << 16;  // instruction descriptor: B is MN-major

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A sequence's rows, checked (conditions to status, which may be NULL); false: nothing of it is computed.
__device__ __forceinline__ bool sequence(const Params& p, int b, int32_t* status, int& row0, int& n) {
  row0 = p.cu[b];
  n = p.cu[b + 1] - row0;
  if (row0 < 0 || n < 0 || row0 > p.total - n || n > p.max_len) {
    set_status(status, FT_DEV_RANGE);
    return false;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const Params p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  extern __shared__ uint8_t prompt_smem[];
  const uint32_t raw = smem_u32(prompt_smem);
  uint8_t* sm = prompt_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ int find[3];  // first token of the CTA's (-1: no work), the sequence's first row, its tokens
  __shared__ int warp_tot[kThreads / 32];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t poison[3][4];  // rows of V that are not finite, by partly visible tile
  auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;

  // ---- which rows: block `want` of all sequences' blocks of tokens, the last ones (which see most) first
  const int per_tile = 128 / p.G, per_cta = p.ntile * per_tile;  // tokens
  const int h = blockIdx.x % p.nkv, want = blockIdx.x / p.nkv;
  {
    auto blocks = [&](int b, int32_t* status, int& row0, int& n) {
      return sequence(p, b, status, row0, n) ? (n + per_cta - 1) / per_cta : 0;
    };
    int32_t* status = blockIdx.x == 0 ? p.status : nullptr;
    if (tid == 0) find[0] = -1;
    if (tid < 12) poison[tid / 4][tid % 4] = 0u;
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0, row0, n;
    for (int b = b0; b < b1; ++b) sum += blocks(b, status, row0, n);
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
        const int nb = blocks(b, nullptr, row0, n);
        if (i < at + nb) {
          find[0] = (i - at) * per_cta, find[1] = row0, find[2] = n;
          break;
        }
        at += nb;
      }
    }
  }
  const uint32_t bar = sm32 + C::kOffBar;
  const uint32_t q_full = bar, s_full = bar + 8, o_full = bar + 24, drained = bar + 40, looked = bar + 48, turn = bar + 72,
                 p_part = bar + 88, full = bar + 136,
                 empty = full + 8 * C::kSlots;
  if (tid == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      for (int k = 0; k < 3; ++k) mbar_init(p_part + 16 * k + 8 * i, 128);
      mbar_init(turn + 8 * i, 1);
      mbar_init(o_full + 8 * i, 1);
    }
    mbar_init(drained, 2);
    for (int i = 0; i < 3; ++i) mbar_init(looked + 8 * i, 32);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 3);  // both issuing warps' products, and the looking warp: it follows every tile, so that none passes it by
    }
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
  const int tok0 = uni(find[0]), row0 = uni(find[1]), n = uni(find[2]);
  const int end = min(tok0 + per_cta, n);                             // this CTA's tokens: tok0 .. end - 1
  const int ntile = tok0 < 0 ? 0 : min(p.ntile, (end - tok0 + per_tile - 1) / per_tile);
  auto tiles_of = [&](int t) { return (min(tok0 + (t + 1) * per_tile, n) + kKeys - 1) / kKeys; };  // position tiles that tile t sees
  const int nkt = ntile > 0 ? tiles_of(ntile - 1) : 0, nkt0 = ntile > 0 ? tiles_of(0) : 0;
  const int part = (tok0 + 1) / kKeys;  // from this tile on (three at most) some row sees a position that another does not
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax: one row per thread
    regs_up<kRegSoftmax>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    if (t < ntile) {
      const int tok = tok0 + t * per_tile + row / p.G;             // (may be behind the last one: not stored)
      const int seen = tok0 + t * per_tile + 32 * (warp & 3) / p.G;  // every row of the warp sees this position
      const int mine = t == 0 ? nkt0 : nkt;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < mine; ++j) {
        if (!all_wait(s_full + 8 * t, j & 1)) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(tmem + lane_base + 128 * t + c, s + c);
        wait_ld();
        if (kKeys * j + kKeys - 1 > seen) {
          const int lim = tok - kKeys * j;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] = c <= lim ? s[c] : 0xFF800000u;
        }
        float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kKeys; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = max3(q[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
        const float mx = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])) * p.scale;
        const bool need = mx > m + kLazy;
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
        const float u = m == -INFINITY ? 0.0f : -m;
        const f32x2 scale2(p.scale, p.scale), u2(u, u);
        f32x2 sum[2] = {f32x2(0.0f, 0.0f), f32x2(0.0f, 0.0f)};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t o[16];
#pragma unroll
          for (int c = 32 * g; c < 32 * g + 32; c += 2) {
            float x0, x1;
            fma2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, u2).get(x0, x1);
            x0 = ex2(x0), x1 = ex2(x1);
            sum[(c / 2) & 1] = add2(sum[(c / 2) & 1], f32x2(x0, x1));
            const __nv_bfloat162 v = __floats2bfloat162_rn(x0, x1);
            o[(c - 32 * g) / 2] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tmem_st16(tmem + lane_base + 128 * t + 16 * g, o);
          if (g > 0) {  // P is handed over in a half and two quarters
            wait_st();
            fence_before();
            mbar_arrive(p_part + 16 * (g - 1) + 8 * t);
          }
        }
        float a, c;
        add2(sum[0], sum[1]).get(a, c);
        l += a + c;
      }
      // a row of V that is not finite, among those that this row sees
      for (int j = part; ok && j < mine; ++j) {
        if (!all_wait(looked + 8 * (j - part), 0)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int lim = tok - kKeys * j - 32 * g;
          const uint32_t bits = poison[j - part][g] & (lim < 0 ? 0u : lim >= 31 ? 0xFFFFFFFFu : (2u << lim) - 1u);
          if (bits) l = __uint_as_float(0x7FC00000u);
        }
      }
      if (ok && !all_wait(o_full + 8 * t, 0)) ok = false;
      if (ok) {
        fence_after();
        const float inv = 1.0f / l;
        // Each four lanes exchange 16-byte pieces, so that they store 64 bytes of a row together (a row a lane
        // takes the load-store unit a cycle a lane: 4.2 thousand cycles for the tile).
        const int quad = lane & 3, r_first = row & ~3;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32], w[4][4];
          tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
          wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v =
                  __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
              w[i][k] = *reinterpret_cast<const uint32_t*>(&v);
            }
#pragma unroll
          for (int x = 2; x > 0; x >>= 1)  // w[i] of lane q goes to w[q] of lane i
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i & x) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool up = quad & x;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i][k] : w[i + x][k], x);
                if (up) w[i][k] = got;
                else w[i + x][k] = got;
              }
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r_first + i, to = tok0 + t * per_tile + r / p.G;
            if (r >= per_tile * p.G || to >= n) continue;
            uint16_t* dst = p.o + (row0 + to) * p.o_stride + (int64_t)(h * p.G + r % p.G) * D + c + 8 * quad;
            if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) dst[2 * k] = (uint16_t)w[i][k], dst[2 * k + 1] = (uint16_t)(w[i][k] >> 16);
            }
          }
        }
      }
    }
  } else {
    regs_down<kRegOther>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- copies
      if (ntile > 0 && lane == 0) {
        const uint32_t q_bytes = (uint32_t)(per_tile * p.G * D * 2);
        mbar_arrive_expect_tx(q_full, ntile * q_bytes);
        for (int t = 0; t < ntile; ++t)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load(sm32 + C::kOffQ + t * C::kTile + c * (128 * 128), &map_q, 64 * c, h * p.G, row0 + tok0 + t * per_tile, q_full);
        int done = 0;
        for (int i = 0; i < 2 * nkt; ++i, ++done) {  // K0 V0 K1 V1 ...
          const int slot = i % C::kSlots, use = i / C::kSlots;
          if (use > 0 && !mbar_wait(empty + 8 * slot, (use - 1) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full + 8 * slot, C::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load(sm32 + C::kOffRing + slot * C::kTile + c * (128 * 128), (i & 1) ? &map_v : &map_k, 64 * c, h, row0 + kKeys * (i >> 1), full + 8 * slot);
        }
        // nothing of these is in flight when the CTA ends
        if (!mbar_wait(q_full, 0)) ok = false;
        for (int i = max(0, done - C::kSlots); i < done; ++i)
          if (!mbar_wait(full + 8 * (i % C::kSlots), (i / C::kSlots) & 1)) ok = false;
      }
    } else if (warp < kLookWarp) {
      // ---------------------------------------------------------- tensor-core issue, a warp for each tile
      constexpr uint32_t id_qk = idesc_bf16(128, kKeys), id_pv = idesc_bf16(128, D) | kBMn;
      const uint32_t lead = lane == 0 ? 1u : 0u, tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = desc_lo(sm32 + C::kOffQ), ring = sm32 + C::kOffRing;
      const int t = warp - kMmaWarp, mine = t == 0 ? nkt0 : nkt;
      const uint32_t ds = tm + 128 * t, d_o = tm + C::kColO + D * t, qa = q_lo + t * (C::kTile >> 4);
      // the last products of Q K^T are issued when the other tile's turn has begun: no gap between the two
      auto qk = [&](int j, auto&& pass) {
        const uint32_t ka = desc_lo(ring + (2 * j) % C::kSlots * C::kTile);
        mma_ss<false>(ds, qa, ka, id_qk, lead);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks) {
          const uint32_t o = ((ks / 4) * (128 * 128) + 32 * (ks % 4)) >> 4;
          if (ks == D / 16 - kPassLeft) pass();
          mma_ss<true>(ds, qa + o, ka + o, id_qk, lead);
        }
        commit(s_full + 8 * t, lead);
      };
      auto pv = [&](int j, int from, int to) {
        const uint32_t va = desc_lo_mn(ring + (2 * j + 1) % C::kSlots * C::kTile);
#pragma unroll
        for (int ks = from; ks < to; ++ks) mma_ts(d_o, ds + 8 * ks, va + ((ks * 2048) >> 4), id_pv, ks > 0 ? 1u : (uint32_t)j, lead);
      };
      auto arrived = [&](int i) { return all_wait(full + 8 * (i % C::kSlots), (i / C::kSlots) & 1); };
      // (a tile that is not there, or that does not see the last positions, lets go of what it leaves out)
      auto release = [&](int i) { commit(empty + 8 * (i % C::kSlots), lead); };
      if (t < ntile) {
        ok = all_wait(q_full, 0) && arrived(0);
        if (ok) {
          fence_after();
          qk(0, [] {});
        }
        // The tiles take the tensor core by turns, tile 0 first: left alone they fall into step, both softmaxes at
        // once and then both tiles' products.
        const bool turns = ntile == 2;
        auto pass = [&] {
          if (turns && lead) mbar_arrive(turn + 8 * (t ^ 1));
        };
        for (int j = 0; ok && j < mine; ++j) {
          release(2 * j);
          ok = arrived(2 * j + 1) && (j < part || all_wait(looked + 8 * (j - part), 0)) && (j + 1 >= mine || arrived(2 * j + 2)) &&
               all_wait(p_part + 8 * t, j & 1) && (!turns || (t == 0 && j == 0) || all_wait(turn + 8 * t, t == 0 ? (j - 1) & 1 : j & 1));
          if (!ok) break;
          fence_after();
          pv(j, 0, 4);
          ok = all_wait(p_part + 16 + 8 * t, j & 1);
          if (!ok) break;
          fence_after();
          pv(j, 4, 6);
          ok = all_wait(p_part + 32 + 8 * t, j & 1);
          if (!ok) break;
          fence_after();
          pv(j, 6, 8);
          release(2 * j + 1);
          if (j + 1 < mine) {
            qk(j + 1, pass);
          } else {
            commit(o_full + 8 * t, lead);
            pass();
          }
        }
        for (int j = mine; ok && t == 0 && j < nkt; ++j) {  // tile 1 goes on alone
          ok = all_wait(turn, (j - 1) & 1);
          pass();
        }
      }
      for (int i = t < ntile ? 2 * mine : 0; ok && i < 2 * nkt; ++i) {
        ok = arrived(i);
        if (ok) release(i);
      }
      // tensor memory is freed only when nothing issued here is in flight
      commit(drained, lead);
      if (!all_wait(drained, 0)) ok = false;
    } else {
      // ---------------------------------------------------------- V tiles that some row sees in part
      for (int i = 0; i < 2 * nkt; ++i) {
        if (!all_wait(full + 8 * (i % C::kSlots), (i / C::kSlots) & 1)) {
          ok = false;
          break;
        }
        const int j = i >> 1;
        if ((i & 1) == 0 || j < part) {
          if (lane == 0) mbar_arrive(empty + 8 * (i % C::kSlots));
          continue;
        }
        uint8_t* v = sm + C::kOffRing + (i % C::kSlots) * C::kTile;
        for (int r = lane; r < kKeys; r += 32) {
          const int key = kKeys * j + r;
          if (key <= tok0) continue;  // every row sees it
          bool clear = key >= n;
          if (!clear) {
            uint32_t acc = 0u;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(v + (c / 8) * (128 * 128) + r * 128 + (((c + lane) & 7) << 4));
              acc = fma_bf16x2(x.x, 0u, acc), acc = fma_bf16x2(x.y, 0u, acc), acc = fma_bf16x2(x.z, 0u, acc), acc = fma_bf16x2(x.w, 0u, acc);
            }
            clear = (acc & 0x7FFF7FFFu) != 0u;
            if (clear) atomicOr(&poison[j - part][r / 32], 1u << (r % 32));
          }
          if (clear)
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c / 8) * (128 * 128) + r * 128 + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        mbar_arrive(looked + 8 * (j - part));
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * (i % C::kSlots));
      }
    }
  }
  if (!ok) set_status(p.status, FT_DEV_TIMEOUT);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

// [rows][heads][D] BF16 with the given stride between rows, in boxes of `tokens` rows x `heads_box` heads x 64 channels.
static bool make_map(CUtensorMap* map, const uint16_t* at, int D, int heads, int64_t rows, int64_t stride, int heads_box, int tokens) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t size[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t step[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)tokens}, each[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(at), size, step, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static cudaError_t launch(Params& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int64_t blocks, cudaStream_t st) {
  static int allowed[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    // the roles' register shares add up to kRegLaunch a thread: a build with fewer would wait for them forever
    cudaFuncAttributes fa = {};
    if (cudaFuncGetAttributes(&fa, prompt_kernel<D>) != cudaSuccess) return cudaErrorInvalidDeviceFunction;
    if (fa.numRegs < kRegLaunch) return cudaErrorInvalidConfiguration;
    allowed[dev] = 1;
  }
  prompt_kernel<D><<<(unsigned)(blocks * p.nkv), kThreads, Cfg<D>::kSmem, st>>>(p, q, k, v);
  return cudaGetLastError();
}

}  // namespace prompt

constexpr int kPromptMaxB = 8192;

}  // namespace ft

extern "C" {

int ft_attn_prompt_bf16(const ft_block_cfg* c, const uint16_t* q_bf16, int64_t q_stride, const uint16_t* k_bf16,
                        int64_t k_stride, const uint16_t* v_bf16, int64_t v_stride, const int32_t* cu_seqlens, int B,
                        int total, int max_len, float scale, uint16_t* o_bf16, int64_t o_stride, int32_t* dev_status,
                        ft_stream stream) {
  const int st = ft_host::check_cfg(c);
  if (st != FT_OK) return st;
  if (B < 1 || total < 0 || max_len < 1 || !(scale > 0.0f) || !(scale < 3e38f)) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  const int D = c->head_dim, G = c->n_q / c->n_kv;
  const int64_t row_q = (int64_t)c->n_q * D, row_k = (int64_t)c->n_kv * D;
  if (!q_bf16 || !k_bf16 || !v_bf16 || !cu_seqlens || !o_bf16 || q_stride < row_q || o_stride < row_q || k_stride < row_k ||
      v_stride < row_k)
    return FT_ERR_INVALID_ARG;
  if (!ft_host::aligned16(q_bf16) || !ft_host::aligned16(k_bf16) || !ft_host::aligned16(v_bf16) || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return FT_ERR_INVALID_ARG;
  if (B > ft::kPromptMaxB || (int64_t)total * G > INT32_MAX) return FT_ERR_UNSUPPORTED;
  // tensor maps hold strides below 2^40 bytes
  if (std::max(q_stride, std::max(k_stride, v_stride)) >= (int64_t)1 << 39) return FT_ERR_UNSUPPORTED;
  const int per_tile = 128 / G;
  // two tiles a CTA, one where all blocks then still run at once
  int sms = ft_host::num_sms();
  if (sms <= 0) sms = 152;
  const int64_t some = std::min(B, total);
  ft::prompt::Params p = {};
  p.ntile = ((int64_t)total / per_tile + some) * c->n_kv > sms ? 2 : 1;
  const int64_t blocks = total / (p.ntile * per_tile) + some;
  if (blocks * c->n_kv > INT32_MAX) return FT_ERR_UNSUPPORTED;
  CUtensorMap q, k, v;
  if (!ft::prompt::make_map(&q, q_bf16, D, c->n_q, total, q_stride, G, per_tile) ||
      !ft::prompt::make_map(&k, k_bf16, D, c->n_kv, total, k_stride, 1, 128) || !ft::prompt::make_map(&v, v_bf16, D, c->n_kv, total, v_stride, 1, 128))
    return FT_ERR_CUDA;
  p.q = q_bf16;
  p.o = o_bf16;
  p.o_stride = o_stride;
  p.cu = cu_seqlens;
  p.status = dev_status;
  p.B = B;
  p.total = total;
  p.max_len = max_len;
  p.nkv = c->n_kv;
  p.G = G;
  p.scale = scale * 1.44269504088896341f;
  const cudaError_t e = D == 128 ? ft::prompt::launch<128>(p, q, k, v, blocks, (cudaStream_t)stream)
                                 : ft::prompt::launch<64>(p, q, k, v, blocks, (cudaStream_t)stream);
  return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
