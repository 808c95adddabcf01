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
// Roles: two warpgroups of softmax (one row per thread, a tile each); a warp that works out the items and of which one
// thread issues the TMA copies of Q, K and V; two that issue the products, one for each tile, which take the tensor core
// by turns
//   PV0(j) QK0(j+1) PV1(j) QK1(j+1) ...
// so that it works for one while the other's softmax runs; and one that looks through the V tiles which some row sees
// in part: rows behind the sequence's end become zeros, and so do rows that are not finite (0 x infinity would reach
// the rows before them), which are noted for the rows that see them.
// The running max moves only when a score passes it by 2^8 (P is BF16, sums are FP32), so O is rarely rescaled.
// Every wait is bounded; a timeout sets FT_DEV_TIMEOUT and the CTA winds down.
//
// Measured, 32 heads over 8 of 128: 8192 tokens 317 us (1735 TFLOP/s of the causal half), 8 prompts of up to 2048 83 us
// (1130), 100 tokens 7.5.  Bound by the tensor core, 2570 cycles a pair of tiles of which it works 2048, and by about
// 6500 cycles a block beside its tiles: query rows in, first S, last P V, rows out, which only half overlap.
#include <cuda.h>

#include <algorithm>

#include "ft_prompt_items.h"
#include "ft_tc.cuh"

namespace ft {

namespace prompt {

using namespace tiles;

constexpr int kThreads = 384, kKeys = 128;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLookWarp = 11;  // (two issuing warps)
constexpr float kLazy = 8.0f;
constexpr int kWorks = 2;  // items known ahead
constexpr int kLooks = 8;  // partly visible tiles of V looked through ahead: more than the ring holds, and one item's, together
constexpr int kPassLeft = 1;  // products of a batch issued behind the end of its turn (1, 2, 3, 5: 344, 349, 360, 371 us for 8192 tokens)
static_assert(kPassLeft > 0 && kPassLeft < 64 / 16, "the turn is passed on in every batch");
// Registers of a thread: softmax twice, the others; the sum over the three warpgroups is what the block is
// launched with, kThreads x kRegLaunch.
constexpr int kRegSoftmax = 208, kRegOther = 88, kRegLaunch = 168;
static_assert(2 * kRegSoftmax + kRegOther <= 3 * kRegLaunch, "more registers than the block has");

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;              // Q, K or V: 128 rows
  static constexpr int kSlots = D == 128 ? 5 : 8;         // of the ring that K and V tiles come through: K0 V0 K1 V1 ...
  static constexpr int kOffQ = 0, kOffRing = 2 * kTile, kOffBar = kOffRing + kSlots * kTile;
  static constexpr int kBars = 512, kSmem = kOffBar + kBars + 1024;  // 1024: alignment slack
  static constexpr int kColO = 256;                       // tensor memory: S0, S1, then O0, O1
};

struct Params {
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

// What a CTA works on: tokens tok0, tok0 + 1, ... of one sequence for KV head h, and what follows from them.
struct Item {
  int tok0, row0, n, h;  // tok0 < 0: no more
  int ntile, nkt, nkt0, part;
  __device__ __forceinline__ Item(const Params& p, int4 w) : tok0(w.x), row0(w.y), n(w.z), h(w.w) {
    const int per_tile = 128 / p.G, end = min(tok0 + p.ntile * per_tile, n);
    ntile = (end - tok0 + per_tile - 1) / per_tile;
    nkt = (end + kKeys - 1) / kKeys;  // position tiles that the last tile of rows sees, and
    nkt0 = (min(tok0 + per_tile, n) + kKeys - 1) / kKeys;  // the first one
    part = (tok0 + 1) / kKeys;  // from this tile on (three at most) some row sees a position that another does not
  }
};

// A place in a ring of N barriers: slot and the parity of its current use.
template <int N>
struct Cursor {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, parity ^= 1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const Params p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  using Ring = Cursor<C::kSlots>;
  extern __shared__ uint8_t prompt_smem[];
  const uint32_t raw = smem_u32(prompt_smem);
  uint8_t* sm = prompt_smem + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sm32 = smem_u32(sm);
  __shared__ __align__(16) int4 work[kWorks];
  __shared__ __align__(16) uint32_t answer[4];  // of the request for another CTA's place
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t poison[kLooks][4];  // rows of V that are not finite, by partly visible tile
  auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  const int per_tile = 128 / p.G;

  const uint32_t bar = sm32 + C::kOffBar;
  const uint32_t q_full = bar, q_empty = bar + 16, s_full = bar + 32, o_full = bar + 48, turn = bar + 64, p_part = bar + 80,
                 work_full = bar + 128, work_empty = work_full + 8 * kWorks, answered = work_empty + 8 * kWorks, drained = answered + 8,
                 looked = drained + 8, full = looked + 8 * kLooks, empty = full + 8 * C::kSlots;
  static_assert(128 + 16 * kWorks + 16 + 8 * kLooks + 16 * C::kSlots <= C::kBars, "barriers");
  if (tid == 32 * kLoadWarp) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(turn + 8 * i, 1);
      for (int k = 0; k < 3; ++k) mbar_init(p_part + 16 * k + 8 * i, 128);
    }
    for (int i = 0; i < kWorks; ++i) {
      mbar_init(work_full + 8 * i, 1);
      mbar_init(work_empty + 8 * i, 8 + 2 + 1);  // the warps of softmax, issue and looking
    }
    mbar_init(answered, 1);
    mbar_init(drained, 2);
    for (int i = 0; i < kLooks; ++i) mbar_init(looked + 8 * i, 32);
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
  griddep_serve();  // (barriers and tensor memory are set up beside the kernel before this one)
  bool ok = true;
  // The k-th item, for a whole warp; tok0 < 0 behind the last one, or where the wait ran out.
  auto take = [&](uint32_t k) {
    const int slot = k % kWorks;
    int4 w = make_int4(-1, 0, 0, 0);
    if (all_wait(work_full + 8 * slot, (k / kWorks) & 1)) w = work[slot];
    else ok = false;
    __syncwarp();
    if (lane == 0) mbar_arrive(work_empty + 8 * slot);
    return make_int4(uni(w.x), uni(w.y), uni(w.z), uni(w.w));
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax: one row per thread
    regs_up<kRegSoftmax>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    uint32_t tiles_done = 0, items_done = 0, looks_done = 0;
    for (uint32_t k = 0; ok; ++k) {
      const int4 got = take(k);
      if (got.x < 0) break;
      const Item w(p, got);
      const uint32_t look0 = looks_done;
      looks_done += w.nkt - w.part;
      if (t >= w.ntile) continue;
      const int tok = w.tok0 + t * per_tile + row / p.G;                     // (may be behind the last one: not stored)
      const int seen = w.tok0 + t * per_tile + 32 * (warp & 3) / p.G;  // every row of the warp sees this position
      const int mine = t == 0 ? w.nkt0 : w.nkt;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < mine; ++j, ++tiles_done) {
        if (!all_wait(s_full + 8 * t, tiles_done & 1)) {
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
      for (int j = w.part; ok && j < mine; ++j) {
        const uint32_t look = look0 + (j - w.part);
        if (!all_wait(looked + 8 * (look % kLooks), (look / kLooks) & 1)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int lim = tok - kKeys * j - 32 * g;
          const uint32_t bits = poison[look % kLooks][g] & (lim < 0 ? 0u : lim >= 31 ? 0xFFFFFFFFu : (2u << lim) - 1u);
          if (bits) l = __uint_as_float(0x7FC00000u);
        }
      }
      if (ok && !all_wait(o_full + 8 * t, items_done & 1)) ok = false;
      ++items_done;
      if (ok) {
        fence_after();
        const float inv = 1.0f / l;
        const int in = row / p.G;
        uint16_t* dst = row >= per_tile * p.G || tok >= w.n ? nullptr : p.o + (w.row0 + tok) * p.o_stride + (int64_t)(w.h * p.G + (row - in * p.G)) * D;
        const uintptr_t low = reinterpret_cast<uintptr_t>(dst);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32], x[16];
          tmem_ld32(tmem + lane_base + C::kColO + D * t + c, o);
          wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            x[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (!dst) continue;
          if ((low & 31u) == 0) {  // whole sectors: half the time of 16-byte pieces
            st_global_v8(dst + c, x);
            st_global_v8(dst + c + 16, x + 8);
          } else if ((low & 15u) == 0) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(dst + c + 2 * i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[c + 2 * i] = (uint16_t)x[i], dst[c + 2 * i + 1] = (uint16_t)(x[i] >> 16);
          }
        }
      }
    }
  } else {
    regs_down<kRegOther>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- what to work on, and copies
      // Item x is (block of tokens, head) x of all sequences' blocks.  With up to 32 sequences (a lane each) the blocks that see most
      // come first: those of the same place in their sequences together, from the last place on (8 prompts of up to 2048:
      // 92 -> 85 us); else each sequence's last ones first.  The grid has a CTA for each; those that run take the places
      // of those that have not begun.
      if (lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
      }
      const int per_cta = p.ntile * per_tile, per = (p.B + 31) / 32, b0 = min(lane * per, p.B), b1 = min(b0 + per, p.B);
      auto blocks = [&](int b, int32_t* status, int& row0, int& n) {
        return sequence(p, b, status, row0, n) ? (n + per_cta - 1) / per_cta : 0;
      };
      int sum = 0, row0 = 0, n = 0;  // (of the lane's sequence, where it has one)
      for (int b = b0; b < b1; ++b) sum += blocks(b, p.status, row0, n);
      auto scan = [&](int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += up;
        }
        return x;
      };
      const int inc = scan(sum), total = __shfl_sync(0xffffffffu, inc, 31);
      ItemWalk walk(__reduce_max_sync(0xffffffffu, sum) - 1);  // (a sequence a lane)
      Ring at;
      uint32_t k = 0, q_uses[2] = {0, 0}, used = 0, asked = 0;
      int x = blockIdx.x;
      for (bool more = true; more;) {
        if (lane == 0) {  // the next one, while this one is worked on
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(answered, 16);
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(answer)),
                       "r"(answered)
                       : "memory");
        }
        int i = x / p.nkv;
        if (i < total) {
          int4 got = make_int4(0, 0, 0, x % p.nkv);
          if (per == 1) {
            const uint32_t some =
                walk.find(i, [&](int level) { return __ballot_sync(0xffffffffu, sum > level); }, [](uint32_t bits) { return __popc(bits); });
            const int l = __fns(some, 0, i - walk.above + 1);
            got.x = walk.level * per_cta, got.y = __shfl_sync(0xffffffffu, row0, l), got.z = __shfl_sync(0xffffffffu, n, l);
          } else {
            i = total - 1 - i;
            const int l = __ffs(__ballot_sync(0xffffffffu, i < inc)) - 1;  // the lane that holds it
            i -= __shfl_sync(0xffffffffu, inc - sum, l);
            for (int b = min(l * per, p.B), b_end = min(b + per, p.B); b < b_end; b += 32) {
              int r = 0, m = 0;
              const int nb = b + lane < b_end ? blocks(b + lane, nullptr, r, m) : 0, up = scan(nb);
              const uint32_t hit = __ballot_sync(0xffffffffu, i < up);
              if (hit) {
                const int f = __ffs(hit) - 1;
                got.x = (i - __shfl_sync(0xffffffffu, up - nb, f)) * per_cta;
                got.y = __shfl_sync(0xffffffffu, r, f), got.z = __shfl_sync(0xffffffffu, m, f);
                break;
              }
              i -= __shfl_sync(0xffffffffu, up, 31);
            }
          }
          if (k >= kWorks && !all_wait(work_empty + 8 * (k % kWorks), (k / kWorks - 1) & 1)) ok = false;
          if (ok && lane == 0) {
            work[k % kWorks] = got;
            mbar_arrive(work_full + 8 * (k % kWorks));
          }
          ++k;
          const Item w(p, got);
          // K0, the query rows, V0 K1 V1 ...: the first tile's slot is free before the query rows' places are (8192 tokens:
          // 324 -> 318 us).  One loop, as what runs once comes from a cold instruction cache.
#pragma unroll 1
          for (int step = 0; ok && step < 2 * w.nkt + 2; ++step) {
            const int t = step - 1, j = step == 0 ? 0 : step - 2;  // query rows of tile t, or K / V tile j
            const bool rows = t == 0 || t == 1;
            if (t == 1 && w.ntile == 1) continue;
            const uint32_t to = rows ? q_full + 8 * t : full + 8 * at.slot, free_at = rows ? q_empty + 8 * t : empty + 8 * at.slot;
            const uint32_t before = rows ? (t == 0 ? q_uses[0] : q_uses[1]) : used >= C::kSlots ? 1u : 0u;
            if (before > 0 && !all_wait(free_at, rows ? (before - 1) & 1 : at.parity ^ 1)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(to, rows ? (uint32_t)(per_tile * p.G * D * 2) : (uint32_t)C::kTile);
              const CUtensorMap* map = rows ? &map_q : (j & 1) ? &map_v : &map_k;
              const uint32_t dst = sm32 + (rows ? C::kOffQ + t * C::kTile : C::kOffRing + at.slot * C::kTile);
              const int head = rows ? w.h * p.G : w.h, first = w.row0 + (rows ? w.tok0 + t * per_tile : kKeys * (j >> 1));
#pragma unroll
              for (int c = 0; c < D / 64; ++c) tma_load(dst + c * (128 * 128), map, 64 * c, head, first, to);
            }
            if (rows) {
              if (t == 0) ++q_uses[0];
              else ++q_uses[1];
            } else {
              at.next();
              ++used;
            }
          }
        }
        // the answer: a CTA that will not run any more, whose place is taken here, or none
        uint32_t taken = 0, next = 0;
        if (all_wait(answered, asked & 1)) {
          asm volatile(
              "{ .reg .pred p; .reg .b128 h; ld.shared.b128 h, [%2];\n"
              "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h; selp.u32 %0, 1, 0, p; mov.u32 %1, 0;\n"
              "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h; }"
              : "=r"(taken), "=r"(next)
              : "r"(smem_u32(answer))
              : "memory");
        } else {
          ok = false;
        }
        ++asked;
        __syncwarp();
        x = uni((int)next);
        more = ok && uni((int)taken) != 0;
      }
      if (ok && (k < kWorks || all_wait(work_empty + 8 * (k % kWorks), (k / kWorks - 1) & 1))) {
        if (lane == 0) {
          work[k % kWorks] = make_int4(-1, 0, 0, 0);
          mbar_arrive(work_full + 8 * (k % kWorks));
        }
      } else {
        ok = false;
      }
      if (!ok) {  // no copy is in flight when the CTA ends
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (q_uses[t] > 0) mbar_wait(q_full + 8 * t, (q_uses[t] - 1) & 1);
        Ring last;
        for (uint32_t i = 0; i < used; ++i, last.next())
          if (i + C::kSlots >= used) mbar_wait(full + 8 * last.slot, last.parity);
      }
    } else if (warp < kLookWarp) {
      // ---------------------------------------------------------- tensor-core issue, a warp for each tile
      constexpr uint32_t id_qk = idesc_bf16(128, kKeys), id_pv = idesc_bf16(128, D) | kBMn;
      const uint32_t lead = lane == 0 ? 1u : 0u, tm = __shfl_sync(0xffffffffu, tmem, 0), ring = sm32 + C::kOffRing;
      const int t = warp - kMmaWarp;
      const uint32_t ds = tm + 128 * t, d_o = tm + C::kColO + D * t, qa = desc_lo(sm32 + C::kOffQ + t * C::kTile);
      // the last products of Q K^T are issued when the other tile's turn has begun: no gap between the two
      auto qk = [&](int slot, auto&& pass) {
        const uint32_t ka = desc_lo(ring + slot * C::kTile);
        mma_ss<false>(ds, qa, ka, id_qk, lead);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks) {
          const uint32_t o = ((ks / 4) * (128 * 128) + 32 * (ks % 4)) >> 4;
          if (ks == D / 16 - kPassLeft) pass();
          mma_ss<true>(ds, qa + o, ka + o, id_qk, lead);
        }
        commit(s_full + 8 * t, lead);
      };
      auto pv = [&](int slot, int j, int from, int to) {
        const uint32_t va = desc_lo_mn(ring + slot * C::kTile);
#pragma unroll
        for (int ks = from; ks < to; ++ks) mma_ts(d_o, ds + 8 * ks, va + ((ks * 2048) >> 4), id_pv, ks > 0 ? 1u : (uint32_t)j, lead);
      };
      auto arrived = [&](const Ring& r) { return all_wait(full + 8 * r.slot, r.parity); };
      auto release = [&](const Ring& r) { commit(empty + 8 * r.slot, lead); };
      Ring at;  // K of the current tile
      uint32_t tiles_done = 0, items_done = 0, looks_done = 0, turns_done = 0;
      for (uint32_t k = 0; ok; ++k) {
        const int4 got = take(k);
        if (got.x < 0) break;
        const Item w(p, got);
        const int mine = t >= w.ntile ? 0 : t == 0 ? w.nkt0 : w.nkt;
        // The tiles take the tensor core by turns, tile 0 first: left alone they fall into step, both softmaxes at
        // once and then both tiles' products.
        const bool turns = w.ntile == 2;
        auto pass = [&] {
          if (turns && lead) mbar_arrive(turn + 8 * (t ^ 1));
        };
        auto my_turn = [&] {
          if (!turns) return true;
          const uint32_t i = turns_done++;
          return t == 0 ? i == 0 || all_wait(turn, (i - 1) & 1) : all_wait(turn + 8, i & 1);
        };
        if (mine > 0) {
          ok = all_wait(q_full + 8 * t, items_done & 1) && arrived(at);
          if (!ok) break;
          fence_after();
          qk(at.slot, [] {});
          if (mine == 1) commit(q_empty + 8 * t, lead);
          ++items_done;
        }
        for (int j = 0; ok && j < mine; ++j, ++tiles_done) {
          release(at);
          Ring v = at;
          v.next();
          at = v;
          at.next();
          const uint32_t look = looks_done + (j - w.part);
          ok = arrived(v) && (j < w.part || all_wait(looked + 8 * (look % kLooks), (look / kLooks) & 1)) && (j + 1 >= mine || arrived(at)) &&
               all_wait(p_part + 8 * t, tiles_done & 1) && my_turn();
          if (!ok) break;
          fence_after();
          pv(v.slot, j, 0, 4);
          ok = all_wait(p_part + 16 + 8 * t, tiles_done & 1);
          if (!ok) break;
          fence_after();
          pv(v.slot, j, 4, 6);
          ok = all_wait(p_part + 32 + 8 * t, tiles_done & 1);
          if (!ok) break;
          fence_after();
          pv(v.slot, j, 6, 8);
          release(v);
          if (j + 1 < mine) {
            qk(at.slot, pass);
            if (j + 2 == mine) commit(q_empty + 8 * t, lead);
          } else {
            commit(o_full + 8 * t, lead);
            pass();
          }
        }
        for (int j = mine; ok && j < w.nkt; ++j) {  // what the other tile sees alone is let go of
          for (int i = 0; ok && i < 2; ++i, at.next()) {
            ok = arrived(at);
            if (ok) release(at);
          }
          ok = ok && my_turn();
          pass();
        }
        looks_done += w.nkt - w.part;
      }
      // tensor memory is freed only when nothing issued here is in flight
      commit(drained, lead);
      if (!all_wait(drained, 0)) ok = false;
    } else {
      // ---------------------------------------------------------- V tiles that some row sees in part
      Ring at;
      uint32_t look = 0;
      for (uint32_t k = 0; ok; ++k) {
        const int4 got = take(k);
        if (got.x < 0) break;
        const Item w(p, got);
        for (int i = 0; i < 2 * w.nkt; ++i, at.next()) {
          if (!all_wait(full + 8 * at.slot, at.parity)) {
            ok = false;
            break;
          }
          const int j = i >> 1;
          if ((i & 1) && j >= w.part) {
            uint8_t* v = sm + C::kOffRing + at.slot * C::kTile;
            if (lane < 4) poison[look % kLooks][lane] = 0u;
            __syncwarp();
            for (int r = lane; r < kKeys; r += 32) {
              const int key = kKeys * j + r;
              if (key <= w.tok0) continue;  // every row sees it
              bool clear = key >= w.n;
              if (!clear) {
                uint32_t acc[4] = {0u, 0u, 0u, 0u};  // zero unless something is infinite or NaN
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                  const uint4 x = *reinterpret_cast<const uint4*>(v + (c / 8) * (128 * 128) + r * 128 + (((c + lane) & 7) << 4));
                  acc[0] = fma_bf16x2(x.x, 0u, acc[0]), acc[1] = fma_bf16x2(x.y, 0u, acc[1]);
                  acc[2] = fma_bf16x2(x.z, 0u, acc[2]), acc[3] = fma_bf16x2(x.w, 0u, acc[3]);
                }
                clear = ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7FFF7FFFu) != 0u;
                if (clear) atomicOr(&poison[look % kLooks][r / 32], 1u << (r % 32));
              }
              if (clear)
                for (int c = 0; c < D / 8; ++c)
                  *reinterpret_cast<uint4*>(v + (c / 8) * (128 * 128) + r * 128 + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            mbar_arrive(looked + 8 * (look % kLooks));
            ++look;
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(empty + 8 * at.slot);
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
  return launch_served(prompt_kernel<D>, dim3((unsigned)(blocks * p.nkv)), dim3(kThreads), Cfg<D>::kSmem, st, 1, p, q, k, v);
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
