// Paged 4-bit KV cache: block tables and slot maps from request lengths, placement
// of new K/V rows through a slot map, and reading rows back.
#include <algorithm>

#include "ft_paged.cuh"

namespace ft {

// ------------------------------------------------------------------ page map
// One cluster of up to kMapCtas CTAs (one launch: a decode step's call is bound by
// its latency).  Every CTA scans all request lengths for itself (B <= 8192: a few
// loads a thread), keeping the prefix sums of rows and of pages taken in shared
// memory; the cluster then meets once, so that outputs may alias the inputs they
// advance (kv_len = ctx_len, free_head_out = free_head), and the CTAs share the
// slots and the new table entries, each found by a binary search.
constexpr int kMapCtas = 8, kMapThreads = 1024, kMapMaxB = 8192;

struct MapParams {
  const int32_t *ctx, *add, *free_pages, *free_head;
  int32_t *table, *head_out, *cu, *kv_len, *slots, *status;
  int B, stride, n_free, n_slots, n_pages, pshift;
};

// Exclusive scan of one value per thread over the CTA; total to every thread.
__device__ __forceinline__ long long block_scan(long long v, long long& total, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const long long w = warp_sums[lane];
    long long winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += up;
    }
    warp_sums[lane] = winc - w;
    if (lane == 31) warp_sums[32] = winc;
  }
  __syncthreads();
  const long long ex = warp_sums[warp] + inc - v;
  total = warp_sums[32];
  __syncthreads();
  return ex;
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

__global__ void __launch_bounds__(kMapThreads, 1) page_map_kernel(const MapParams p) {
  extern __shared__ int32_t map_smem[];
  __shared__ long long warp_sums[33];
  __shared__ int bad;
  const int tid = threadIdx.x, B = p.B;
  int32_t* cu = map_smem;            // [B + 1] first row of each request
  int32_t* pg = cu + B + 1;          // [B + 1] first page taken by each request
  int32_t* ctx_s = pg + B + 1;       // [B] history length, -1: not served
  if (tid == 0) bad = 0;
  const int head = p.free_head ? *p.free_head : 0;
  const long long avail = (head >= 0 && head <= p.n_free) ? p.n_free - head : 0;
  const int per = (B + kMapThreads - 1) / kMapThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  const long long cap = (long long)p.stride << p.pshift;  // positions of one table row
  const int round = (1 << p.pshift) - 1;
  long long rows = 0, need = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = p.ctx[b], a = p.add[b];
    rows += max(a, 0);
    if (c >= 0 && a >= 0 && (long long)c + a <= cap)
      need += (((long long)c + a + round) >> p.pshift) - (((long long)c + round) >> p.pshift);
  }
  long long n_rows, n_need;
  long long r = block_scan(rows, n_rows, warp_sums);
  long long q = block_scan(need, n_need, warp_sums);
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = p.ctx[b], a = p.add[b];
    cu[b] = (int)min(r, (long long)INT32_MAX);
    pg[b] = (int)min(q, (long long)INT32_MAX);
    r += max(a, 0);
    bool served = c >= 0 && a >= 0 && (long long)c + a <= cap;
    if (served) {
      const long long n = (((long long)c + a + round) >> p.pshift) - (((long long)c + round) >> p.pshift);
      q += n;
      if (n > 0) {
        served = q <= avail;
        if (served) taken = (int)q;
      }
    }
    ctx_s[b] = served ? c : -1;
    if (!served) bad = FT_DEV_CAPACITY;  // same value from every thread
  }
  // pages taken: the largest prefix sum that a served request reached
  __syncthreads();
  long long most = taken;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if ((tid & 31) == 0) warp_sums[tid >> 5] = most;
  if (tid == 0) {
    cu[B] = (int)min(n_rows, (long long)INT32_MAX);
    pg[B] = (int)min(n_need, (long long)INT32_MAX);
  }
  __syncthreads();
  for (int w = 0; w < 32; ++w) most = max(most, warp_sums[w]);
  const int n_taken = (int)most, total = min(cu[B], p.n_slots);
  cluster_arrive();
  cluster_wait();  // every CTA has read the lengths and the head

  const int first = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
  if (blockIdx.x == 0) {
    for (int b = tid; b <= B; b += kMapThreads) p.cu[b] = cu[b];
    for (int b = b0; b < b1; ++b) p.kv_len[b] = ctx_s[b] < 0 ? 0 : ctx_s[b] + (cu[b + 1] - cu[b]);
    if (tid == 0) {
      if (p.head_out) *p.head_out = head + n_taken;
      if (n_rows > p.n_slots || head < 0 || head > p.n_free) bad |= FT_DEV_RANGE;
      if (bad) set_status(p.status, bad);
    }
  }
  // page id of the free list's entry i, or -1 (and a flag) where it is no page
  auto fresh = [&](int i) {
    const int id = p.free_pages[head + i];
    if (id >= 0 && id < p.n_pages) return id;
    set_status(p.status, FT_DEV_RANGE);
    return -1;
  };
  for (int i = first; i < n_taken; i += step) {
    const int b = last_not_above(pg, B, i);
    const int old = (int)(((long long)ctx_s[b] + round) >> p.pshift);
    if (ctx_s[b] >= 0) p.table[(size_t)b * p.stride + old + (i - pg[b])] = fresh(i);
  }
  for (int i = first; i < p.n_slots; i += step) {
    int slot = -1;
    if (i < total) {
      const int b = last_not_above(cu, B, i), c = ctx_s[b];
      if (c >= 0) {
        const int pos = c + (i - cu[b]), ip = pos >> p.pshift, old = (int)(((long long)c + round) >> p.pshift);
        const int id = ip < old ? p.table[(size_t)b * p.stride + ip] : fresh(pg[b] + ip - old);
        if (id >= 0 && id < p.n_pages)
          slot = (id << p.pshift) + (pos & round);
        else
          set_status(p.status, FT_DEV_RANGE);
      }
    }
    p.slots[i] = slot;
  }
}

// ------------------------------------------------------------------ placement
// D / 4 lanes per (row, head, K or V): each lane owns the four channels of one
// 16-bit word of the entry (paged_fwht's ownership), so the rotated row is
// quantised and stored without passing through shared memory.
template <int D>
__global__ void __launch_bounds__(256) append_paged_kernel(const uint16_t* __restrict__ k, int64_t k_stride,
                                                           const uint16_t* __restrict__ v, int64_t v_stride,
                                                           const int32_t* __restrict__ slots,
                                                           uint8_t* __restrict__ pages, PagedLayout L, int64_t nvec,
                                                           int hb, float norm, int32_t* status) {
  constexpr int LV = D / 4;
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t vec = gid / LV;
  const int lane = (int)(gid % LV), g = lane & 7, j = lane >> 3;
  const bool live = vec < nvec;
  const int which = (int)(vec & 1);
  const int64_t th = vec >> 1;
  const int h = (int)(th % L.nkv);
  const int64_t t = th / L.nkv;
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int slot = -1;
  if (live) {
    slot = slots[t];
    const uint16_t* src = which ? v + t * v_stride : k + t * k_stride;
    src += h * D + 32 * j + g;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = bf16_bits_to_f32(src[8 * e]);
  }
  paged_fwht<D>(x, hb, norm);
  float am = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  bool bad = !(fabsf(x[0]) <= 3e38f && fabsf(x[1]) <= 3e38f && fabsf(x[2]) <= 3e38f && fabsf(x[3]) <= 3e38f);
#pragma unroll
  for (int o = LV / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const uint16_t sb = quant_scale_bits(am);
  const float s = bf16_bits_to_f32(sb);
  int c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = max((int)quant_code(x[e], s) - 8, -7);
  const uint32_t w = paged_pack(c[0], c[1], c[2], c[3]);
  if (!live || slot == -1) return;
  if (slot < 0 || (slot >> L.pshift) >= L.npages) {
    if (lane == 0) set_status(status, FT_DEV_RANGE);
    return;
  }
  if (bad) set_status(status, FT_DEV_RANGE);
  const int p = slot & (L.psize - 1);
  uint8_t* blk = pages + paged_block(L, slot >> L.pshift, h);
  const uint32_t off = which ? L.voff + paged_v_word<D>(p, g, j) : paged_k_word<D>(p, g, j);
  *reinterpret_cast<uint16_t*>(blk + off) = (uint16_t)w;
  if (lane == 0) *reinterpret_cast<uint16_t*>(blk + L.soff + 4 * p + 2 * which) = sb;
}

// Rows of the given slots as values in the model basis: decoded, rotated back,
// rounded to BF16.
template <int D>
__global__ void __launch_bounds__(256) read_paged_kernel(const uint8_t* __restrict__ pages, PagedLayout L,
                                                         const int32_t* __restrict__ slots,
                                                         uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                                                         int64_t nvec, int hb, float norm, int32_t* status) {
  constexpr int LV = D / 4;
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t vec = gid / LV;
  const int lane = (int)(gid % LV), g = lane & 7, j = lane >> 3;
  const bool live = vec < nvec;
  const int which = (int)(vec & 1);
  const int64_t th = vec >> 1;
  const int h = (int)(th % L.nkv);
  const int64_t t = th / L.nkv;
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (live) {
    const int slot = slots[t];
    if (slot >= 0 && (slot >> L.pshift) < L.npages) {
      const int p = slot & (L.psize - 1);
      const uint8_t* blk = pages + paged_block(L, slot >> L.pshift, h);
      const uint32_t off = which ? L.voff + paged_v_word<D>(p, g, j) : paged_k_word<D>(p, g, j);
      const uint32_t w = *reinterpret_cast<const uint16_t*>(blk + off);
      const float s = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(blk + L.soff + 4 * p + 2 * which));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = paged_value(w, e) * s;
    } else if (slot != -1 && lane == 0) {
      set_status(status, FT_DEV_RANGE);
    }
  }
  paged_fwht<D>(x, hb, norm);
  if (!live) return;
  uint16_t* dst = (which ? v_out : k_out) + th * D + 32 * j + g;
#pragma unroll
  for (int e = 0; e < 4; ++e) dst[8 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(x[e]));
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
  if (smem > 48 * 1024 && attr_smem[dev] < smem) {
    const int most = (3 * ft::kMapMaxB + 2) * 4;
    if (cudaFuncSetAttribute(ft::page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return FT_ERR_CUDA;
    attr_smem[dev] = most;
  }
  cudaLaunchConfig_t cfg = {};
  // a CTA for every 1024 rows, as a power of two up to the cluster's limit
  int ctas = 1;
  while (ctas < ft::kMapCtas && ctas * ft::kMapThreads < n_slots) ctas *= 2;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(ft::kMapThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ft::page_map_kernel, p) == cudaSuccess ? FT_OK : FT_ERR_CUDA;
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
  const ft::PagedLayout L = ft::paged_layout(*c, n_pages, page_size);
  const int64_t nvec = (int64_t)total * c->n_kv * 2, blocks = (nvec * (c->head_dim / 4) + 255) / 256;
  if (blocks > (int64_t)INT32_MAX) return FT_ERR_UNSUPPORTED;
  const auto kernel = c->head_dim == 128 ? ft::append_paged_kernel<128> : ft::append_paged_kernel<64>;
  kernel<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(k_bf16, k_stride, v_bf16, v_stride, slots,
                                                             static_cast<uint8_t*>(pages), L, nvec, c->had_block,
                                                             ft::paged_norm(c->had_block), dev_status);
  return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

int ft_kv_read_paged_int4(const ft_block_cfg* c, const void* pages, int n_pages, int page_size, const int32_t* slots,
                          int total, uint16_t* k_out, uint16_t* v_out, int32_t* dev_status, ft_stream stream) {
  const int st = ft_host::check_paged(c, pages, n_pages, page_size);
  if (st != FT_OK) return st;
  if (total < 0) return FT_ERR_INVALID_ARG;
  if (total == 0) return FT_OK;
  if (!slots || !k_out || !v_out) return FT_ERR_INVALID_ARG;
  const ft::PagedLayout L = ft::paged_layout(*c, n_pages, page_size);
  const int64_t nvec = (int64_t)total * c->n_kv * 2, blocks = (nvec * (c->head_dim / 4) + 255) / 256;
  if (blocks > (int64_t)INT32_MAX) return FT_ERR_UNSUPPORTED;
  const auto kernel = c->head_dim == 128 ? ft::read_paged_kernel<128> : ft::read_paged_kernel<64>;
  kernel<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(static_cast<const uint8_t*>(pages), L, slots, k_out, v_out,
                                                             nvec, c->had_block, ft::paged_norm(c->had_block),
                                                             dev_status);
  return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

}  // extern "C"
