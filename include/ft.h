/*
 * ft.h -- C ABI of the INT4-weight / Hadamard-rotated INT4-KV decode block.
 *
 * One Llama-style Transformer block, one new token per request, on one GPU
 * (sm_103a).  The operations follow the statement of the problem on the pages
 * "FuTransformer: FP8 prefill and INT4 decode for Llama-style inference on
 * Hopper" (summary page on onedev.kr, sections "어떻게 동작하나" / how it
 * works, "무엇과 다른가" / what differs, "전제와 한계" / premises and limits).
 *
 * Conventions (all calls):
 *  - Every pointer argument is a DEVICE pointer unless stated otherwise.  The
 *    caller allocates and owns all memory; the library never allocates.
 *  - Calls are asynchronous on the caller's stream and return an ft_status
 *    code.  Host-side argument checks happen before anything is enqueued; a
 *    failed check enqueues nothing.
 *  - Conditions only the device can see (a position beyond the cache capacity,
 *    an activation outside the FP16 range, a bounded wait that ran out) are
 *    OR-ed into the caller's int32 device status word (may be NULL) as
 *    FT_DEV_* bits; read it after synchronising.  Kernels never trap.
 *  - No exception or abort crosses this boundary.
 */
#ifndef FT_H_
#define FT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st *ft_stream;

/* ---- status codes ------------------------------------------------------ */
enum {
  FT_OK = 0,
  FT_ERR_INVALID_ARG = -1, /* NULL/misaligned pointer, bad size, overlap    */
  FT_ERR_UNSUPPORTED = -2, /* shape or option this build does not implement */
  FT_ERR_WORKSPACE = -3,   /* workspace or packed buffer too small          */
  FT_ERR_CAPACITY = -4,    /* batch larger than the cache's max_batch       */
  FT_ERR_CUDA = -5         /* a CUDA runtime call failed (launch, attrs)    */
};

/* bits OR-ed into the device status word */
enum {
  FT_DEV_CAPACITY = 1, /* pos[b] (+T) outside [0, max_ctx): that request skipped */
  FT_DEV_TIMEOUT = 2,  /* a bounded pipeline wait ran out; outputs invalid       */
  FT_DEV_RANGE = 4     /* an activation exceeded the FP16 operand range          */
};

/* activation dtypes of the block input/output */
enum { FT_BF16 = 0, FT_F32 = 1 };

/* decode-weight formats (ft_block_cfg.weight_format): INT4 codes, or E4M3 codes
 * (summary page, "전제와 한계": E4M3 decode weights as the FP8 variant of the
 * decode path), both with one BF16 scale per (output row, 128 inputs) */
enum { FT_WFMT_INT4 = 0, FT_WFMT_E4M3 = 1 };

/* ---- configuration ------------------------------------------------------ */
typedef struct {
  int32_t hidden;    /* H; multiple of 128                                      */
  int32_t n_q;       /* query heads; multiple of n_kv, n_q / n_kv <= 8          */
  int32_t n_kv;      /* KV heads                                               */
  int32_t head_dim;  /* d in {64, 128}                                          */
  int32_t inter;     /* SwiGLU intermediate I; multiple of 128                  */
  int32_t w_group;   /* weight group along the input axis; must be 128         */
  int32_t had_block; /* Hadamard block h_b: power of two dividing d (1 = none) */
  int32_t kv_group;  /* channels per KV scale; must equal head_dim             */
  float rms_eps;     /* RMSNorm epsilon                                        */
  float rope_base;   /* RoPE base                                              */
  int32_t weight_format; /* FT_WFMT_INT4 (0) or FT_WFMT_E4M3                    */
} ft_block_cfg;

/* Projection roles.  Weights are given in the logical row-major [N_out, K_in]
 * orientation:  QKV [(n_q+2 n_kv) d, H] (q rows, then k, then v);
 * O [H, n_q d];  GATEUP [2 I, H] (I gate rows, then I up rows);  DOWN [H, I]. */
typedef enum { FT_W_QKV = 0, FT_W_O = 1, FT_W_GATEUP = 2, FT_W_DOWN = 3 } ft_wrole;

/* Describes a status code; never NULL. */
const char *ft_status_string(int status);

/* Host-only check of a configuration (FT_OK, FT_ERR_INVALID_ARG, FT_ERR_UNSUPPORTED). */
int ft_validate_cfg(const ft_block_cfg *cfg);

/* Logical shape [n_out, k_in] of a role's weight matrix (host pointers out). */
int ft_weight_shape(const ft_block_cfg *cfg, int role, int32_t *n_out, int32_t *k_in);

/* ---- weights ------------------------------------------------------------
 * Packing (summary page, "어떻게 동작하나": the fixed RMSNorm gain is folded
 * into the weights before quantisation, W' = gamma W; "무엇과 다른가": INT4
 * values with group scales applied after accumulation, stored in the order the
 * kernel consumes them).  For each output row o and each group of 128
 * consecutive input channels: W'[o,i] = W[o,i] * gamma[i] (FP32 product),
 * s = bf16_rne(amax / 7), code = clamp(rne(W' / s), -8, 7) + 8 (FP32
 * decisions; s = 0 gives code 8).  The packed buffer is opaque: 128-row blocks,
 * 16-row tiles, per (tile, group) 1024 bytes of nibbles in the tensor-core
 * fragment order the decode kernels read, followed by the 16 BF16 scales. */

/* Bytes of one packed role in the configuration's weight format: INT4 codes
 * P/2 + scales P/64, or E4M3 codes P + scales P/64, for P = N_out * K_in. */
size_t ft_packed_weight_bytes(const ft_block_cfg *cfg, int role);

/* W: FP32 [N_out, K_in] row-major.  gamma: FP32 [K_in] or NULL (treated as 1);
 * use gamma_attn for QKV and gamma_ffn for GATEUP.  packed: >= 16-byte aligned,
 * packed_bytes >= ft_packed_weight_bytes().  Overwrites packed entirely.
 * cfg->weight_format must be FT_WFMT_INT4 (else FT_ERR_INVALID_ARG). */
int ft_pack_weights_int4(const ft_block_cfg *cfg, int role, const float *W, const float *gamma,
                         void *packed, size_t packed_bytes, ft_stream stream);

/* Inverse view for tests: codes uint8 [N_out, K_in] in [0,15] (value code-8)
 * and scales as BF16 bits [N_out, K_in/128], logical orientation. */
int ft_unpack_weights_int4(const ft_block_cfg *cfg, int role, const void *packed, uint8_t *codes,
                           uint16_t *scales_bf16, ft_stream stream);

/* E4M3 decode weights (summary page, "전제와 한계"; the abstract page compares
 * the INT4 decode path with an FP8 one).  For each output row o and group of 128
 * consecutive inputs: W'[o,i] = W[o,i] * gamma[i] (FP32), s = bf16_rne(amax /
 * 448), code = E4M3(W' / s) rounded to nearest, ties to even, saturating at
 * +-448, the sign of zero kept (FP32 division; s = 0 gives code 0x00).  Same
 * row-tile-major layout as INT4 with 2048 bytes of codes per (tile, group) in
 * the tensor-core fragment order, then the 16 BF16 scales.  Arguments as for
 * ft_pack_weights_int4; cfg->weight_format must be FT_WFMT_E4M3. */
int ft_pack_weights_e4m3(const ft_block_cfg *cfg, int role, const float *W, const float *gamma, void *packed,
                         size_t packed_bytes, ft_stream stream);

/* Inverse layout transform of ft_pack_weights_e4m3 (for tests): codes as E4M3
 * bytes [N_out, K_in] and scales as BF16 bits [N_out, K_in/128]. */
int ft_unpack_weights_e4m3(const ft_block_cfg *cfg, int role, const void *packed, uint8_t *codes,
                           uint16_t *scales_bf16, ft_stream stream);

/* ---- KV cache -----------------------------------------------------------
 * One layer's cache for max_batch requests x n_kv heads x max_ctx positions.
 * Entry (request, head, position) holds d/2 bytes of K nibbles, d/2 bytes of V
 * nibbles and one BF16 scale each for K and V (kv_group = d), addressed by
 * offset(request, head, position, channel) (summary page, "어떻게 동작하나":
 * direct placement, no dense K/V tensors).  Within an entry the nibbles are
 * permuted into the tensor-core fragment order of the attention kernel; the
 * buffer is opaque to callers. */

size_t ft_kv_cache_bytes(const ft_block_cfg *cfg, int max_batch, int max_ctx);

/* Append T tokens per request (summary page, "무엇과 다른가": block-diagonal
 * Hadamard rotation of the new K and V, then INT4 quantisation with BF16
 * scales; H is the normalised Sylvester matrix of order had_block).
 * k_bf16, v_bf16: BF16 bits [B, T, n_kv, d] (post-RoPE).  pos: device int32
 * [B], first position of request b.  Positions pos[b]..pos[b]+T-1 are written;
 * a request with pos[b] < 0 or pos[b]+T > max_ctx is skipped and sets
 * FT_DEV_CAPACITY.  B <= max_batch or FT_ERR_CAPACITY. */
int ft_kv_append_int4(const ft_block_cfg *cfg, void *cache, int max_batch, int max_ctx,
                      const uint16_t *k_bf16, const uint16_t *v_bf16, const int32_t *pos, int B,
                      int T, int32_t *dev_status, ft_stream stream);

/* Append packed variable-length requests: the K/V rows the prefill side
 * produces for a batch of prompts of different lengths, placed straight at
 * offset(request, head, position, channel) (summary page, "어떻게 동작하나":
 * the QKV epilogue writes the KV cache directly; requests of different lengths
 * are packed).  The prefill GEMM itself is not part of this library; this call
 * is its placement step, with the same rotation and quantiser as
 * ft_kv_append_int4.
 *   k_bf16, v_bf16: BF16 bits [total, n_kv, d] (post-RoPE), the rows of request
 *     0, then request 1, ... back to back.
 *   cu_seqlens: device int32 [B + 1], the prefix sums of the request lengths
 *     (cu_seqlens[0] = 0, cu_seqlens[B] = total, non-decreasing); request b
 *     owns rows cu_seqlens[b] .. cu_seqlens[b+1]-1 (a zero-length request owns
 *     none).
 *   pos: device int32 [B], the first position written for request b.
 * Row cu_seqlens[b] + t goes to position pos[b] + t of request b.  A request
 * whose positions fall outside 0 .. max_ctx-1 is skipped and sets
 * FT_DEV_CAPACITY; a map that is not such a prefix sum writes nothing and sets
 * FT_DEV_RANGE.  B <= max_batch or FT_ERR_CAPACITY; total = 0 enqueues nothing. */
int ft_kv_append_ragged_int4(const ft_block_cfg *cfg, void *cache, int max_batch, int max_ctx,
                             const uint16_t *k_bf16, const uint16_t *v_bf16, const int32_t *cu_seqlens,
                             const int32_t *pos, int B, int total, int32_t *dev_status, ft_stream stream);

/* Inverse view for tests: positions [0, len) of requests [0, B).  codes uint8
 * [B, n_kv, len, d] in logical channel order; scales BF16 bits [B, n_kv, len, 1]. */
int ft_kv_unpack_int4(const ft_block_cfg *cfg, const void *cache, int max_batch, int max_ctx, int B,
                      int len, uint8_t *k_codes, uint8_t *v_codes, uint16_t *k_scales,
                      uint16_t *v_scales, ft_stream stream);

/* ---- paged KV cache -----------------------------------------------------
 * One layer's cache as a pool of pages that requests share: page i holds
 * page_size positions (16, 32, 64 or 128) of every KV head, and a request's
 * block table names its pages in order.  A slot is page * page_size + offset.
 * Rotation and quantiser are those of ft_kv_append_int4 (codes -7..7; -8 never
 * occurs), so a row has the same codes and scales in either cache.  Layout of a
 * page (P = page_size, d = head_dim): n_kv head blocks of P (d + 4) bytes, each
 *   P K entries of d/2 bytes, P/2 V entries of d bytes (positions 2i, 2i + 1),
 *   P pairs of BF16 (K scale, V scale).
 * Values are sign and magnitude, four to a 16-bit word; word (g, j) of a
 * position, g < 8, j < d/32, holds channels 32 j + g + 8 e, e = 0..3, with
 * magnitudes at bits 0, 3, 8, 11 and signs at bits 15, 14, 7, 6.  Its byte is
 *   K, offset p:  p d/2 + (g / 2) d/8 + 4 j + 2 (g % 2)
 *   V, pair i:    i d + (g XOR turn(i)) d/8 + 4 j + 2 (offset % 2),
 *                 turn(i) = 2 (i % 4) for d = 128, 4 ((i / 2) % 2) for d = 64.
 * The pool is 16-byte aligned; all offsets are 64-bit. */

/* Bytes of a pool of n_pages pages; 0 for an invalid configuration. */
size_t ft_kv_pages_bytes(const ft_block_cfg *cfg, int n_pages, int page_size);

/* Block tables, slot map and prefix sums of one step, built on the device from
 * the requests' lengths (no host round trip; can be captured and replayed).
 *   ctx_len, new_len: int32 [B], tokens that request b has in the cache and
 *     tokens that it adds.
 *   block_table: int32 [B, table_stride]; entries of pages that already hold
 *     tokens (ceil(ctx_len / page_size) of them) are read, those of the pages
 *     added are written, the others are left as they are.
 *   free_pages: int32 [n_free]; the pages added are free_pages[head], head + 1,
 *     ... in request order, with head = *free_head (NULL: 0).
 *   free_head_out: int32, head + pages taken (NULL: not written).
 *   cu_seqlens: int32 [B + 1], prefix sums of new_len (2^31 - 1 where they pass
 *     that).  kv_len: int32 [B], ctx_len + new_len.
 *   slots: int32 [n_slots]; slot of row i (request b, position ctx_len[b] + i -
 *     cu_seqlens[b]); -1 for rows behind the last one.
 * kv_len may be ctx_len and free_head_out may be free_head (advanced in place);
 * no other arguments may overlap.  A request with a negative length, more
 * positions than its table row holds (or than 2^31 - 1), or whose new pages end
 * behind the free list sets FT_DEV_CAPACITY and is not served: its rows get slot
 * -1, its kv_len is 0 (also where that is ctx_len) and its table row is left alone
 * (pages are counted in request order, also those of requests that did not get
 * them).  More rows than n_slots, a head outside [0, n_free] or a page outside
 * [0, n_pages) set FT_DEV_RANGE; such rows are dropped (slot -1).  B <= 8192, else
 * FT_ERR_UNSUPPORTED. */
int ft_kv_page_map(int page_size, int n_pages, const int32_t *ctx_len, const int32_t *new_len, int B,
                   int32_t *block_table, int table_stride, const int32_t *free_pages, int n_free,
                   const int32_t *free_head, int32_t *free_head_out, int32_t *cu_seqlens, int32_t *kv_len,
                   int32_t *slots, int n_slots, int32_t *dev_status, ft_stream stream);

/* Rotate, quantise and place `total` rows at their slots.  k_bf16, v_bf16: BF16
 * bits, row t at t * stride (strides in elements, >= n_kv d; a view of the fused
 * projection's output works), [n_kv, d] inside a row, post-RoPE.  slots: int32
 * [total]; -1 skips the row, any other slot outside the pool sets FT_DEV_RANGE
 * and skips it.  The slots of one call must be distinct.  A row whose rotated
 * values are not finite sets FT_DEV_RANGE; what it stores is not defined. */
int ft_kv_append_paged_int4(const ft_block_cfg *cfg, void *pages, int n_pages, int page_size, const uint16_t *k_bf16,
                            int64_t k_stride, const uint16_t *v_bf16, int64_t v_stride, const int32_t *slots, int total,
                            int32_t *dev_status, ft_stream stream);

/* Reads rows back as values in the model basis (decoded, the rotation undone,
 * rounded to BF16): k_out, v_out BF16 bits [total, n_kv, d], 16-byte aligned.  Slot -1 gives zeros;
 * any other slot outside the pool gives zeros and sets FT_DEV_RANGE. */
int ft_kv_read_paged_int4(const ft_block_cfg *cfg, const void *pages, int n_pages, int page_size, const int32_t *slots,
                          int total, uint16_t *k_out, uint16_t *v_out, int32_t *dev_status, ft_stream stream);

/* Attention of the new tokens of B requests over the paged cache (their own K/V
 * appended before): prompts, chunks of prompts, drafts of a few tokens and single
 * tokens, in any mixture.  Token i of request b (row cu_seqlens[b] + i) is at
 * position kv_len[b] - n_b + i, n_b = cu_seqlens[b + 1] - cu_seqlens[b], and
 * attends to positions 0 .. its own:
 *   o = H softmax(scale * (H q) . K^) V^,   query head h reads KV head h / G.
 * q_bf16, o_bf16: BF16 bits, row t at t * stride (elements, >= n_q d), [n_q, d]
 * inside a row, q post-RoPE; o may be q where the strides are equal.  A token at
 * a negative position (kv_len < n_b) sees nothing and gets zeros.  Rows behind
 * cu_seqlens[B] are left as they are.  max_q: an upper bound of n_b; it picks the
 * kernel, one for all requests of the call, and sizes the launch (single tokens over long
 * caches beside a long prompt are faster in a call of their own).  B <= 8192, total_q n_q / n_kv < 2^31,
 * B n_kv (table_stride page_size / 64 + 8) < 2^31 and, with more than 32 rows (below),
 * total_q n_q / 256 + B n_kv < 2^31, else FT_ERR_UNSUPPORTED.
 * Arithmetic: q rounded to FP16 after the rotation (|q scale log2(e)| < 1023, else
 * FT_DEV_RANGE), codes exact, softmax weights rounded to FP16 below the products,
 * sums and statistics in FP32 (with many rows, below, the sums over positions enter
 * the rotation back as two BF16 numbers each, 2^-17).  V scales that lie within a
 * factor 2^100 of each other, none below 2^-100 (smaller ones count as that), are
 * weighed against each other without loss: farther apart, weights whose product with
 * the V scale is under 2^-126 of the row's largest are lost.  An entry whose V scale is
 * 0 has no values, only a weight, kept beside V scales from 2^-70 to 2^40.  With more
 * than 32 rows (tokens x heads of a group) K and V are decoded to FP16 in groups of 32
 * positions, and scales less than 2^-15 of their group's largest are rounded.  Entries
 * behind a token's position may hold anything else; a row that sees one with a scale
 * that is not finite, or 2^110 and more, is NaN (none is for scales below 2^109), and no
 * other row is touched.  What a request's rows are does not depend on the other requests
 * of the call, up to the order of FP32 sums and the kernel that max_q picks.
 * Device conditions: cu_seqlens not ascending within [0, total_q], or n_b > max_q:
 * FT_DEV_RANGE, that request's rows are not written; a kv_len that is negative,
 * longer than table_stride pages or above 2^31 - 257: FT_DEV_CAPACITY, zeros; a
 * page outside the pool: FT_DEV_RANGE, its positions count as masked.
 * The workspace (16-byte aligned) holds partial results during the call only; calls
 * that may run at the same time need one each. */
size_t ft_attn_paged_workspace_bytes(const ft_block_cfg *cfg, int B, int total_q, int max_q);
int ft_attn_paged_int4(const ft_block_cfg *cfg, const void *pages, int n_pages, int page_size, const uint16_t *q_bf16,
                       int64_t q_stride, const int32_t *cu_seqlens, const int32_t *kv_len, const int32_t *block_table,
                       int table_stride, int B, int total_q, int max_q, float scale, uint16_t *o_bf16, int64_t o_stride,
                       void *workspace, size_t ws_bytes, int32_t *dev_status, ft_stream stream);

/* Attention of drafted tokens that form a tree: ft_attn_paged_int4 with a mask among the new tokens.
 * Token i of request b (row cu_seqlens[b] + i) has its entry at position kv_len[b] - n_b + i (its own
 * K/V appended before) and sees all positions before kv_len[b] - n_b, and new token j < n_b where bit
 * j % 32 of tree_mask[(cu_seqlens[b] + i) mask_stride + j / 32] is set; bits from n_b on are ignored.
 * tree_mask: uint32, row i at i * mask_stride words, ceil(max_q / 32) of them read.  Any pattern will do
 * (a token that sees itself and its ancestors; all of a block; none): a row that sees nothing gets zeros.
 * A token whose entry would be at a negative position has none; bits that name it are ignored.  The position
 * that a token is rotated to (its depth in the tree) need not be that of its entry: see
 * ft_kv_append_rope_paged_int4.  Everything else (arithmetic, device conditions, workspace) is as there, and so are the
 * limits; with R = min(max_q, total_q) n_q / n_kv > 16 also B n_kv ceil(R / 256) (table_stride page_size / 64 + 18),
 * B n_kv R and total_q n_q stay below 2^31 - 128, else FT_ERR_UNSUPPORTED. */
size_t ft_attn_tree_workspace_bytes(const ft_block_cfg *cfg, int B, int total_q, int max_q);
int ft_attn_tree_paged_int4(const ft_block_cfg *cfg, const void *pages, int n_pages, int page_size,
                            const uint16_t *q_bf16, int64_t q_stride, const int32_t *cu_seqlens, const int32_t *kv_len,
                            const int32_t *block_table, int table_stride, const uint32_t *tree_mask, int64_t mask_stride,
                            int B, int total_q, int max_q, float scale, uint16_t *o_bf16, int64_t o_stride,
                            void *workspace, size_t ws_bytes, int32_t *dev_status, ft_stream stream);

/* Moves entries inside the pool, of all KV heads: for each request b < B and j < n, the entry at slot
 * src_slots[b n + j] goes to slot dst_slots[b n + j], bit for bit (the accepted branch of a tree to
 * consecutive positions).  The moves of one request happen at once: all its entries are read before
 * any is written, so their slots may overlap.  A slot of -1 on either side skips the move; any other slot outside the pool
 * sets FT_DEV_RANGE and skips it.  The destinations must be distinct, and no other request's sources.
 * src_slots, dst_slots: int32 [B, n]; n <= 256, else FT_ERR_UNSUPPORTED. */
int ft_kv_move_paged_int4(const ft_block_cfg *cfg, void *pages, int n_pages, int page_size, const int32_t *src_slots,
                          const int32_t *dst_slots, int B, int n, int32_t *dev_status, ft_stream stream);

/* ---- rows of the fused projection ----------------------------------------
 * q, k: BF16 bits as the projection leaves them (pre-RoPE), row t at t * stride (elements), [heads, d]
 * inside a row; views of the fused projection's output work, at any alignment.  In FP32:
 *   y = gamma * x / sqrt(mean x^2 + cfg->rms_eps) per head (gamma: FP32 [d]; NULL: y = x),
 *   z_i = y_i cos a - y_(i+d/2) sin a,  z_(i+d/2) = y_(i+d/2) cos a + y_i sin a,  i < d/2,
 *   a = positions[t] cfg->rope_base^(-2i/d),
 * the pairing, the frequencies and the reduction of the angles being the decode block's: a turn's fraction a
 * position, computed in FP64, times the position, modulo one turn without a loss.  The angle's error is that of
 * the fraction, |position| 2^-54 max(1, 1 / rope_base) turns (2^-23 at position 2^31), and FP32's below.
 * positions: int32 [total], any values (tokens of a tree share them).  With a norm, |x| < 2^60. */

/* q_out, k_out: z rounded once to BF16, rows at their own strides; an output may be its input where the
 * strides are equal.  q with q_out, or k with k_out, may be NULL: left out. */
int ft_qk_norm_rope_bf16(const ft_block_cfg *cfg, const uint16_t *q_bf16, int64_t q_stride, const uint16_t *k_bf16,
                         int64_t k_stride, const float *gamma_q, const float *gamma_k, const int32_t *positions, int total,
                         uint16_t *q_out, int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride, ft_stream stream);

/* ft_kv_append_paged_int4 of z (k) and of v as it is: k is normalised, rotated to its position, rotated by H
 * and quantised without a rounding in between, and placed at its slot with v.  Slots as there; the rotation's
 * position need not be the slot's.  q_bf16 not NULL: z (q) goes to q_out as in ft_qk_norm_rope_bf16, also of
 * rows whose slot is -1. */
int ft_kv_append_rope_paged_int4(const ft_block_cfg *cfg, void *pages, int n_pages, int page_size, const uint16_t *k_bf16,
                                 int64_t k_stride, const uint16_t *v_bf16, int64_t v_stride, const float *gamma_k,
                                 const int32_t *positions, const int32_t *slots, int total, const uint16_t *q_bf16,
                                 int64_t q_stride, const float *gamma_q, uint16_t *q_out, int64_t q_out_stride,
                                 int32_t *dev_status, ft_stream stream);

/* Causal attention of whole prompts over their own rows (post-RoPE BF16, not quantised): sequence b owns rows
 * cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q, k, v and o, and its row i attends to its rows 0 .. i:
 *   o_i = sum_j softmax_j(scale q_i . k_j) v_j,   query head h reads KV head h / G.
 * q, o: [total, n_q, d], k, v: [total, n_kv, d] at their strides (elements); q, k and v at 16-byte
 * boundaries with strides of a multiple of 8, else FT_ERR_INVALID_ARG; o may be q where the strides are equal.  Rows that no
 * sequence owns are left as they are.  max_len: an upper bound of the lengths, which are checked against it.
 * Arithmetic: BF16 products, FP32 sums, maxima and statistics, weights rounded to BF16 below the second
 * product (2^-8 each).  A row that sees a v which is not finite is not finite in the channels concerned (it
 * may be NaN in all of them).  A row with a score that is NaN or +infinity is NaN; a score of -infinity (an
 * infinite value in k, q of the other sign) is a weight of 0.  Rows that do not see such a k or v, and other
 * sequences, are not touched.
 * Device conditions: cu_seqlens not ascending within [0, total], or a length above max_len: FT_DEV_RANGE, that
 * sequence's rows are not written.  B <= 8192, total n_q / n_kv < 2^31, strides below 2^39, else
 * FT_ERR_UNSUPPORTED. */
int ft_attn_prompt_bf16(const ft_block_cfg *cfg, const uint16_t *q_bf16, int64_t q_stride, const uint16_t *k_bf16,
                        int64_t k_stride, const uint16_t *v_bf16, int64_t v_stride, const int32_t *cu_seqlens, int B,
                        int total, int max_len, float scale, uint16_t *o_bf16, int64_t o_stride, int32_t *dev_status,
                        ft_stream stream);

/* ---- the decode block ---------------------------------------------------
 * One token per request b < B at position pos[b] (= L_b, its history length):
 *   rho1 = (mean x^2 + eps)^-1/2;  [q;k;v] = rho1 * W'_qkv x      (row factor
 *      applied after the projection's accumulation, "어떻게 동작하나")
 *   RoPE(q, k) at L_b;  k~ = H k, v~ = H v quantised and written at L_b
 *   q~ = H q;  per query head h (KV head h / G, no head expansion,
 *      "전제와 한계"): softmax over positions 0..L_b of q~.k^/sqrt(d) against
 *      the INT4 cache (split across CTAs and merged for long contexts,
 *      "무엇과 다른가"), o = H o~ (inverse rotation)
 *   h1 = x + W_o o;  rho2 = (mean h1^2 + eps)^-1/2;
 *   a = silu(rho2 W'_g h1) * (rho2 W'_u h1);  out = h1 + W_down a.
 * The new token's K/V are written before attending; attention covers
 * positions 0..pos[b] inclusive; the caller advances pos.
 * x_in, x_out: [B, H] of act_dtype (FT_BF16 bits or FT_F32), must not overlap.
 * Arithmetic: tensor-core FP16 operands (codes exact, activations rounded to
 * FP16), FP32 accumulation, epilogues and softmax.  Activations must stay
 * within the FP16 range (|x| < 65504; FT_DEV_RANGE otherwise).
 * The projection weights are in cfg->weight_format (INT4 or E4M3 codes).
 * 1 <= B <= min(32, max_batch); larger B -> FT_ERR_UNSUPPORTED. */
typedef struct {
  const void *qkv, *o, *gateup, *down; /* each from the pack call of cfg->weight_format */
} ft_layer_weights;

size_t ft_decode_workspace_bytes(const ft_block_cfg *cfg, int B, int max_ctx);

int ft_decode_block(const ft_block_cfg *cfg, const ft_layer_weights *w, void *cache, int max_batch,
                    int max_ctx, const void *x_in, void *x_out, int act_dtype, const int32_t *pos,
                    int B, void *workspace, size_t ws_bytes, int32_t *dev_status, ft_stream stream);

/* Stage selection for ft_decode_block_stages (bit mask). */
enum {
  FT_STAGE_PREP = 1,  /* input -> FP16 operand, sums of squares, zero counters */
  FT_STAGE_QKV = 2,   /* QKV projection (x rho1)                             */
  FT_STAGE_ATTN = 4,  /* RoPE, rotation, cache write, split-KV attention     */
  FT_STAGE_O = 8,     /* O projection + residual                              */
  FT_STAGE_MID = 16,  /* h1 -> gate/up operand, sums of squares, down acc.   */
  FT_STAGE_GU = 32,   /* gate/up projection + SwiGLU                          */
  FT_STAGE_DOWN = 64, /* down projection + residual -> x_out                  */
  FT_STAGE_ALL = 127
};

/* Runs a subset of the block's stages on a workspace left by a previous full
 * call with the same arguments (each stage reads what the earlier stages
 * wrote there).  Used to time one stage alone; FT_STAGE_ALL equals
 * ft_decode_block. */
int ft_decode_block_stages(const ft_block_cfg *cfg, const ft_layer_weights *w, void *cache,
                           int max_batch, int max_ctx, const void *x_in, void *x_out, int act_dtype,
                           const int32_t *pos, int B, void *workspace, size_t ws_bytes,
                           int32_t *dev_status, unsigned stage_mask, ft_stream stream);

/* Byte offsets of intermediate tensors inside the workspace (host struct out),
 * for tests:  qkv FP32 [B, (n_q+2n_kv) d] (the projection before rho1 and
 * RoPE);  rho1 FP32 [B];  o FP16, n_q d values per request (attention output
 * after the inverse rotation);  h1 FP32 [B, H];  a FP16, I values per request
 * (SwiGLU output).  o and a are stored in the projections' grouped operand
 * layout: [inputs / 64][B][64], i.e. the B requests' values of each half group
 * of 64 inputs together (one 128-byte row per request); within a request's 64
 * values the order is 0,1,8,9,2,3,10,11,4,5,12,13,6,7,14,15 per 16 inputs,
 * inputs 8..15 of each 16 hold value / 16, and the 8 runs of 8 stored values
 * are permuted: run r is stored at position r XOR (request mod 8). */
typedef struct {
  size_t qkv, rho1, o, h1, a;
  int32_t n_split; /* split-KV chunks per (request, KV head) */
} ft_ws_layout;

int ft_decode_workspace_layout(const ft_block_cfg *cfg, int B, int max_ctx, ft_ws_layout *out);

/* How ft_decode_block partitions one projection (role FT_W_*) for this batch
 * on the current device (148 SMs assumed when no device is visible): ctas
 * launched; rows per set (row_tiles x 16); warps per CTA; 8-token column tiles;
 * whole = 1 when every CTA owns whole sets (no split along the inputs);
 * tensor_core = 1 for the tcgen05 kernel of batches 17-32 (128-row sets, the
 * contraction on the fifth-generation tensor cores), 0 for the streaming
 * mma.sync kernel of batches 1-16; ring stages, groups (128 inputs) per stage
 * and dynamic shared memory per CTA in bytes. */
typedef struct {
  int32_t ctas, row_tiles, warps, col_tiles, whole, tensor_core, stages, groups_per_stage, smem_bytes;
} ft_gemv_info;
int ft_decode_plan_info(const ft_block_cfg *cfg, int B, int max_ctx, int role, ft_gemv_info *out);

/* ---- full decode step helpers (BF16, not INT4) ----------------------------
 * A complete Llama-style decode step is: embedding gather, the decode block
 * per layer (FT_F32 residual between layers), final RMSNorm, LM head (summary
 * page, "전제와 한계": the full Llama-3.1-8B step at batch 1). */

/* x_out[b, :] = table[tokens[b], :] widened to FP32.  table: BF16 bits [V, H];
 * tokens: device int32 [B]; x_out: FP32 [B, H].  A token outside [0, V) gives a
 * zero row and sets FT_DEV_RANGE. */
int ft_embed_bf16(const uint16_t *table, const int32_t *tokens, float *x_out, int B, int V, int H,
                  int32_t *dev_status, ft_stream stream);

/* Final RMSNorm on its own (ft_lm_head_bf16 applies it fused):
 * z[b, :] = bf16(gamma * rho_b * x[b, :]), rho_b = (mean x[b, :]^2 + eps)^-1/2.
 * x: FP32 [B, H]; gamma: FP32 [H]; z_out: BF16 bits [B, H]. */
int ft_rmsnorm_bf16(const float *x, const float *gamma, uint16_t *z_out, int B, int H, float eps,
                    ft_stream stream);

/* Copies the device status word that the calls above OR their asynchronous
 * FT_DEV_* conditions into to *host_out, after waiting for `stream` (every
 * call enqueued before it has finished).  FT_OK, or FT_ERR_CUDA if the copy or
 * the wait fails. */
int ft_read_device_status(const int32_t *dev_status, int32_t *host_out, ft_stream stream);

/* logits[b, v] = sum_k W[v, k] * z[b, k] with z = gamma * rho(x_b) * x_b,
 * rho = (mean x^2 + eps)^-1/2.  x: FP32 [B, H]; gamma: FP32 [H]; W: BF16 bits
 * [V, H] (16-byte aligned); logits: FP32 [B, V] (overwritten; every element
 * is written once, no accumulation, so repeated calls give the same bits).
 * B <= 32 and H a multiple of 128, else FT_ERR_UNSUPPORTED.  Tokens run in
 * chunks of min(8, 160 KiB / (4 H)) (one launch each, W streamed once per
 * chunk).  z enters the tensor cores as a BF16 (hi, lo) pair. */
int ft_lm_head_bf16(const float *x, const float *gamma, const uint16_t *W, float *logits, int B, int V, int H,
                    float eps, ft_stream stream);

/* Log probabilities of given tokens from logits [N, V] (FT_F32 or FT_BF16, row i at
 * i * row_stride elements, e.g. those of ft_lm_head_bf16):
 *   logprob[i] = x[target] - log sum exp x;   entropy[i] = - sum p log p (nats);
 *   rank[i] = number of tokens before the target, by value and then lower index;
 *   top_ids, top_logprobs [N, top_k]: the top_k first ones in that order.
 * Any output pointer may be NULL (top_k = 0: no alternatives); targets may be NULL
 * where neither logprob nor rank is asked for.  Masked logits are -infinity.  A
 * target of -1 means none: logprob 0, rank -1; any other outside [0, V) gives NaN
 * and -1 and sets FT_DEV_RANGE.  A row with a NaN or +infinity, or with nothing above
 * -infinity, gives NaN (ids and rank -1) and sets FT_DEV_RANGE.  All sums in FP32.
 * top_k <= min(32, V) and V <= 2^30, else FT_ERR_UNSUPPORTED. */
int ft_logprobs(const void *logits, int dtype, int64_t row_stride, int N, int V, const int32_t *targets, int top_k,
                float *logprob, float *entropy, int32_t *rank, int32_t *top_ids, float *top_logprobs,
                int32_t *dev_status, ft_stream stream);

/* ft_decode_block without a caller-provided workspace.  The FuTransformer paper
 * has no counterpart to this call; it exists for callers that cannot allocate
 * device memory when they run a step (a pool or allocation policy that forbids
 * new device allocations after start-up, a host that hands over only input and
 * output buffers, or a loop that must not pay for an allocation).  The scratch
 * space is a fixed 48 MiB device array inside this library, held by every GPU
 * that loads it until the process exits; problems needing more (see
 * ft_decode_workspace_bytes; the 70B layer shape at batch 32 needs about
 * 33 MiB) return FT_ERR_WORKSPACE and enqueue nothing.  No memory is allocated
 * by this call.  The array is shared by all calls on a device and keeps the
 * previous call's contents (the block clears what it needs itself); calls that
 * overlap on the GPU race on it.  The first call on each device looks up the
 * array's address (cudaGetSymbolAddress) with that device current; make that
 * first call before any stream capture.  The address is kept for the process's
 * life: do not use this call on a device after cudaDeviceReset in the same
 * process.  Arguments and results are otherwise those of ft_decode_block. */
int ft_decode_block_static_ws(const ft_block_cfg *cfg, const ft_layer_weights *w, void *cache, int max_batch,
                              int max_ctx, const void *x_in, void *x_out, int act_dtype, const int32_t *pos, int B,
                              int32_t *dev_status, ft_stream stream);

/* Number of kernels one ft_decode_block call with batch B launches: 7 for
 * INT4 weights and B <= 16; 9 where the projections run on the tensor cores
 * (17 <= B <= 32, or E4M3 weights at any batch) and two small kernels finish
 * gate/up (SwiGLU) and the block output from the per-piece partial sums.
 * 0 for an invalid configuration. */
int ft_decode_block_launches(const ft_block_cfg *cfg, int B);

/* Programmatic dependent launch between the block's kernels (default on).
 * Returns the previous setting. */
int ft_set_pdl(int enabled);

#ifdef __cplusplus
}
#endif

#endif /* FT_H_ */
