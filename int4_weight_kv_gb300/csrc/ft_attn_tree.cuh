// What the kernels of attention for draft trees share (ft_attn_tree.cu, ft_attn_tree_few.cu): how the work is shared out, the
// kernel that goes before them (prefix sums, query rows) and the one that joins their partials.
//
// The work is the list of (request, block of up to 256 rows, head, 128 positions) in this order; each CTA takes an equal,
// contiguous share of it whatever the lengths are.  A share's segment is its part of one (request, block, head); it costs
// about as much beside its positions as some units of them do, so each counts that many more, ahead of its first.  Every
// segment leaves (max, sum, accumulator) partials, joined in the order of the shares.
#pragma once

#include <algorithm>

#include "ft_attn_paged.cuh"
#include "ft_tc.cuh"

namespace ft {
namespace tree {

using namespace tiles;

constexpr int kRows = 256, kKeys = 128;
// Units that a share has at least.  2 / 3 / 6 / 12 / 24 (us): one tree of 7 tokens over 64 positions 11.5 / 11.4 / 15.3 / 23.0 /
// 38.9, over 4096 14.8 / 15.7 / 19.7 / 26.2 / 41.8, 32 of up to 7 over up to 200 18.5 / 18.5 / 23.6 / 27.4 / 39.5, over up to 4096
// 44.5 but for 24 (58.3); one of 64 tokens over 300 17.4 / 19.7 / 22.2 / 25.8 / 34.1, over 32768 85.5 for all.  So 2 or 3
// would do better by small trees and worse by none of these.
constexpr int kMinShare = 6;
constexpr int kPartHead = 8;  // a partial: 4 unused, max, sum, 2 unused, accumulator (at a 32-byte boundary)

// The rows of a head and a request lie one behind the other, in q as in `first`.  Partials: of a segment that begins its
// (request, block, head), by the row's place in q; of one that goes on with it, by CTA.
struct Split {
  int4* req;    // [B + 1] of a request: the units before it, first row, tokens (0: none, or malformed), length; then (all units)
  uint16_t* q;  // the rotated queries as FP16 operand rows, [n_kv][total_q][G][D], channels in the order of the cache's words
  float *first, *more;
  int ctas, seg, rows;  // CTAs; a segment's cost beside its positions, in units; rows of a CTA in `more`
  float odd, up;        // factors of the queries' channels c % 16 >= 8, and of the accumulators
};

// Units of a request: blocks of kRows rows, for each head of each `seg` and one for each 128 positions and 128 rows.
struct Units {
  int rows, keys, full, seg;  // rows and position tiles of the request, blocks of kRows rows
  int pair, last, total;      // units of one head of a full block, and of the last block if it is not full; all
  __device__ __forceinline__ Units(const AttnPagedParams& p, int n, int kv, int seg_) : seg(seg_) {
    rows = n * p.G;
    keys = max(1, (kv + kKeys - 1) / kKeys);
    full = rows / kRows;
    pair = seg + 2 * keys;
    const int rest = rows % kRows;
    last = rest == 0 ? 0 : seg + (rest > 128 ? 2 : 1) * keys;
    total = p.L.nkv * (full * pair + last);
  }
  __device__ __forceinline__ int weight(int block) const { return block < full || rows % kRows > 128 ? 2 : 1; }
  // first tile of positions at or behind unit `at` of its (block, head)
  __device__ __forceinline__ int tile(int block, int at) const {
    const int w = weight(block);
    return at <= seg ? 0 : min((at - seg + w - 1) / w, keys);
  }
};
// Shares of `units` on `ctas` CTAs: as many as there are CTAs, none of fewer than kMinShare units but the only one
// (of two at least, so that each holds the beginning of a 256-row tile).
__device__ __forceinline__ int shares_of(int units, int ctas) { return max(min(units / kMinShare, ctas), 1); }
__device__ __forceinline__ int share_begin(int units, int ctas, int c) { return c * (units / ctas) + min(c, units % ctas); }
__device__ __forceinline__ int share_of(int units, int ctas, int u) {
  const int per = units / ctas, rem = units % ctas, cut = rem * (per + 1);
  return u < cut ? u / (per + 1) : rem + (u - cut) / max(per, 1);
}
// A CTA's share as one of its warps walks through it, segment by segment.
struct Share {
  int b, off, left;  // request (behind the last one or < 0: no more), place in its units, units left
  int4 req;          // its record
  // (all lanes; the records of up to 32 requests are loaded together with the sum)
  __device__ __forceinline__ void begin(const AttnPagedParams& p, const Split& sp, int lane) {
    int4 r = __ldcg(sp.req + min(lane, p.B - 1));
    const int units = __ldcg(&sp.req[p.B].x);
    const int shares = shares_of(units, gridDim.x), c = min((int)blockIdx.x, shares), u = share_begin(units, shares, c);
    left = share_begin(units, shares, min(c + 1, shares)) - u;
    b = 0;  // the last request whose units begin at or before u
    if (p.B <= 32) {
      b = __popc(__ballot_sync(0xffffffffu, lane > 0 && lane < p.B && r.x <= u));
    } else {  // by steps of 32 candidates
      int st = 1;
      while (st * 32 < p.B) st *= 32;
      for (; st; st /= 32)
        for (int all = 32; all == 32 && b < p.B;) {
          const int i = min(b + (lane + 1) * st, p.B);
          all = __popc(__ballot_sync(0xffffffffu, i < p.B && __ldcg(sp.req + i).x <= u));
          b += st * all;
        }
      r = __ldcg(sp.req + b);
    }
    const int from = p.B <= 32 ? b : 0;
    req.x = __shfl_sync(0xffffffffu, r.x, from), req.y = __shfl_sync(0xffffffffu, r.y, from);
    req.z = __shfl_sync(0xffffffffu, r.z, from), req.w = __shfl_sync(0xffffffffu, r.w, from);
    off = u - req.x;
  }
  // The next segment: tiles j0 .. j1 - 1 of head h of a block of request b.
  __device__ __forceinline__ bool next(const AttnPagedParams& p, const Split& sp, int& block, int& h, int& j0, int& j1) {
    while (left > 0 && b < p.B) {
      const Units x(p, req.z, req.w, sp.seg);
      if (req.z == 0 || off >= x.total) {
        off = 0;
        if (++b < p.B) req = __ldcg(sp.req + b);
        continue;
      }
      const int span = p.L.nkv * x.pair;
      block = x.full == 0 ? 0 : min(off / span, x.full);
      const int in = off - block * span, len = block < x.full ? x.pair : x.last;
      h = in / len;
      const int at = in - h * len, go = min(left, len - at);
      j0 = x.tile(block, at), j1 = x.tile(block, at + go);
      off += go, left -= go;
      if (j0 < j1) return true;  // (else the share ends in what the segment costs beside its positions)
    }
    return false;
  }
};
// What the host checks: no call's units or rows pass 2^31.
inline bool units_fit(const AttnPagedParams& p) {
  const int64_t blocks = ((int64_t)p.max_q * p.G + kRows - 1) / kRows, keys = (int64_t)p.table_stride * p.L.psize / kKeys + 1;
  return blocks * (16 + 2 * keys) <= INT32_MAX / ((int64_t)p.B * p.L.nkv) &&
         (int64_t)p.B * p.L.nkv <= INT32_MAX / std::max<int64_t>(1, (int64_t)p.max_q * p.G) &&
         (int64_t)p.total_q * p.L.nkv * p.G <= INT32_MAX - 128;
}

// The prefix sums (the first CTA), and the query rows rotated and rounded to FP16 (the others): D / 32 lanes a row, 32
// channels a lane.
//
// The kernel behind this one reads tables, masks and pages as constants (__ldg, ld.global.nc), which a kernel that lives
// beside its predecessor must not do.  It may here: this kernel lets it begin only behind its own wait, when all that came
// before the call is complete, and writes nothing of them itself.  What it does write (records, queries) is read by L2
// loads.  A kernel for attention that began beside the caller's kernels would have to read all of it by ordinary loads.
constexpr int kPrepThreads = 128;  // (four warps)
template <int D>
__global__ void __launch_bounds__(kPrepThreads) tree_prepare_kernel(const AttnPagedParams p, const Split sp) {
  constexpr int LV = D / 32, R = 32 / LV, NJ = D / 32;
  griddep_serve();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0) {
    __shared__ int sums[kPrepThreads / 32];
    const int per = (p.B + kPrepThreads - 1) / kPrepThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    auto units_of = [&](int b, int32_t* status, int4& r) {
      r = make_int4(0, 0, 0, 0);
      if (!attn_request(p, b, status, r.y, r.z, r.w) || r.z == 0) r.z = 0;
      return r.z == 0 ? 0 : Units(p, r.z, r.w, sp.seg).total;
    };
    int sum = 0;
    int4 r;
    for (int b = b0; b < b1; ++b) sum += units_of(b, p.status, r);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += sums[w];
    for (int b = b0; b < b1; ++b) {
      const int units = units_of(b, nullptr, r);
      r.x = at;
      sp.req[b] = r;
      at += units;
    }
    if (b1 == p.B && b0 < b1) sp.req[p.B] = make_int4(at, 0, 0, 0);
    return;
  }
  const int nq = p.L.nkv * p.G;
  const int row = ((int)(blockIdx.x - 1) * (kPrepThreads / 32) + warp) * R + lane / LV, rows = p.total_q * nq;
  const bool in = row < rows;
  const int tok = in ? row / nq : 0, h = in ? row - tok * nq : 0, j = lane % LV, kvh = h / p.G;
  // Rows before the first request's and behind the last one's (a call padded to a fixed number of rows) may hold anything:
  // they are rotated as the others are, read by nobody, and not reported.  (Where the requests do not ascend from the one
  // end to the other, that is reported, with the same condition.)
  const bool owned = tok >= __ldcg(p.cu) && tok < __ldcg(p.cu + p.B);
  const uint16_t* src = p.q + tok * p.q_stride + (int64_t)h * D + 32 * j;
  f32x2 v[16];
  if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(src)[i];
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) v[4 * i + c] = f32x2(__uint_as_float(y[c] << 16), __uint_as_float(y[c] & 0xFFFF0000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = f32x2(bf16_bits_to_f32(src[2 * i]), bf16_bits_to_f32(src[2 * i + 1]));
  }
  paged_fwht<D>(v, p.hb);
  if (!in) return;
  const float f0 = p.qscale * p.norm;
  uint32_t over = 0u;  // stays zero unless a value is infinite or NaN in FP16
  uint4* to = reinterpret_cast<uint4*>(sp.q + ((int64_t)(kvh * p.total_q + tok) * p.G + (h - kvh * p.G)) * D);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, c;
      v[q + 4 * e].get(a, c);
      const float f = (e & 1) ? f0 * sp.odd : f0;
      const __half2 hv = __floats2half2_rn(a * f, c * f);
      o[e] = *reinterpret_cast<const uint32_t*>(&hv);
      over = hfma2(o[e], 0u, over);
    }
    to[j + NJ * q] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (owned && (over & 0x7FFF7FFFu) != 0u) set_status(p.status, FT_DEV_RANGE);
}

// Joins the parts of each row, W = 1 or 4 warps a row.
template <int D, int W>
__global__ void __launch_bounds__(128) tree_join_kernel(const AttnPagedParams p, const Split sp, int groups) {
  constexpr int PW = D + kPartHead;
  const int g = blockIdx.x % groups, bh = blockIdx.x / groups, h = bh % p.L.nkv, b = bh / p.L.nkv;
  const int r = W == 1 ? 4 * g + (threadIdx.x >> 5) : g;
  griddep_serve();
  const int units = __ldcg(&sp.req[p.B].x);
  const int4 req = __ldcg(sp.req + b);
  if (r >= req.z * p.G) return;
  const Units x(p, req.z, req.w, sp.seg);
  const int shares = shares_of(units, sp.ctas);
  const int block = r / kRows;
  const int u0 = req.x + block * p.L.nkv * x.pair + h * (block < x.full ? x.pair : x.last) + sp.seg;
  const int c0 = share_of(units, shares, u0), c1 = share_of(units, shares, u0 + x.weight(block) * (x.keys - 1));
  const int tok = r / p.G, hh = h * p.G + (r - tok * p.G);
  const float *first = sp.first + ((int64_t)(h * p.total_q + req.y) * p.G + r) * PW + 4, *more = sp.more + ((int64_t)(c0 + 1) * sp.rows + (r - block * kRows)) * PW + 4;
  join_row<D, W>(p, c1 - c0 + 1, [&](int i) { return i == 0 ? first : more + (int64_t)(i - 1) * sp.rows * PW; }, sp.up,
                 p.o + (int64_t)(req.y + tok) * p.o_stride + (int64_t)hh * D);
}

// Bytes of the workspace; the pointers into it (given at 16 bytes, used from the next 32 on).
inline size_t split_bytes(int B, int64_t q_rows, int D, int ctas, int rows) {
  return align_up((size_t)(B + 1) * 16, 256) + (size_t)q_rows * D * 2 + ((size_t)ctas * rows + (size_t)q_rows) * (D + kPartHead) * 4 + 16;
}
inline Split split_of(void* workspace, int B, int64_t q_rows, int D, int ctas, int rows) {
  Split sp = {};
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~(uintptr_t)31);
  sp.req = reinterpret_cast<int4*>(ws);
  ws += align_up((size_t)(B + 1) * 16, 256);
  sp.q = reinterpret_cast<uint16_t*>(ws);
  ws += (size_t)q_rows * D * 2;  // (a multiple of 128)
  sp.more = reinterpret_cast<float*>(ws);
  sp.first = sp.more + (size_t)ctas * rows * (D + kPartHead);
  sp.ctas = ctas;
  sp.rows = rows;
  return sp;
}
template <int D>
cudaError_t launch_prepare(const AttnPagedParams& p, const Split& sp, cudaStream_t st) {
  const int per = kPrepThreads / 32 * (32 / (D / 32));
  const int64_t q_rows = (int64_t)p.total_q * p.L.nkv * p.G;
  return launch_served(tree_prepare_kernel<D>, dim3((unsigned)(1 + (q_rows + per - 1) / per)), dim3(kPrepThreads), 0, st, 1, p, sp);
}
template <int D>
cudaError_t launch_join(const AttnPagedParams& p, const Split& sp, cudaStream_t st) {
  // Four warps a row where a row may have more than twelve partials (a warp loads eight at once).  One warp / this rule /
  // four (us): one tree of 4 tokens, 64 heads over 8, over 32768 positions 35.1 / 32.1 / 32.1, of 64 85.4 / 85.5 / 93.8; 32 of
  // up to 7 over up to 4096 44.6 / 44.6 / 54.6.  From 6 partials on: 93.8 for the tree of 64; from 24 on: as from 12.
  const int rows = p.max_q * p.G;
  const bool wide = ((int64_t)p.total_q * p.G / kRows + std::min(p.B, p.total_q)) * p.L.nkv * 12 < sp.ctas;
  const int groups = wide ? rows : (rows + 3) / 4;
  return launch_served(wide ? tree_join_kernel<D, 4> : tree_join_kernel<D, 1>, dim3((unsigned)(p.B * p.L.nkv * groups)), dim3(128), 0, st, 1, p, sp,
                       groups);
}
inline int num_sms() {
  const int sms = ft_host::num_sms();
  return sms > 0 ? sms : 152;
}

}  // namespace tree
}  // namespace ft
