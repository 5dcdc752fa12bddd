/*
 * bitq_lm.h -- the operators that stand between the packed linear layers of a
 * decoder: a paged key-value cache (page tables and slot maps built on the
 * GPU, cache writes, attention of one new token per request), the residual
 * update of a block with its norms, and the int8 matrix product for layers
 * kept in 8 bits.
 *
 * Conventions are those of bitq.h: the caller owns every buffer, the library
 * allocates nothing, every argument is checked before anything is enqueued
 * (a negative bitq_status and bitq_last_error() on error, nothing written),
 * launches are asynchronous on the given stream (a hipStream_t as void*,
 * NULL = the null stream) and never synchronize.  A non-gfx950 device gives
 * BITQ_E_UNSUPPORTED, a launch failure BITQ_E_DEVICE.  Lengths, page tables
 * and slots live on the GPU, so their values cannot be checked on the host;
 * each call says what its kernels do with values outside their range (none
 * of them makes a kernel read or write outside its buffers).
 */
#ifndef BITQ_LM_H
#define BITQ_LM_H

#include <stddef.h>
#include <stdint.h>

#include "bitq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ======================================================= paged cache */

typedef enum {
    BITQ_KV_BF16 = 0,  /* rows in bf16 */
    BITQ_KV_INT8 = 1   /* rows as int8 codes with one fp32 scale per row */
} bitq_kv_dtype;

/*
 * Geometry of the key-value cache of one layer: a pool of `pages` pages of
 * `page` tokens.  A slot is a token's place in the pool,
 * slot = page_index * page + offset.
 *
 * Layout of the cache buffer (Dp = head_dim rounded up to 32, the elements
 * past head_dim zero; sections at multiples of 256 bytes, in this order):
 *   K  [pages][kv_heads][page][Dp]       bf16 or int8
 *   V  [pages][kv_heads][page/8][Dp][8]  bf16 or int8: 8 consecutive tokens of
 *                                        one element lie together (the order in
 *                                        which the attention's matrix
 *                                        instructions take values)
 *   ks f32 [pages][kv_heads][page]       int8 only: the rows' scales
 *   vs f32 [pages][kv_heads][page]       int8 only
 * A row of int8 codes q with scale d stands for the values q d; d = amax/127
 * and q = clamp(rint(x fl32(127/amax)), -127, 127) as in bitq_quantize_act.
 */
typedef struct {
    int32_t kv_heads;  /* 1 .. 1024 */
    int32_t head_dim;  /* 1 .. 256 */
    int32_t page;      /* tokens per page: a power of two, 8 .. 1024 */
    int32_t pages;     /* pages of the pool; pages * page < 2^31 */
    int32_t dtype;     /* bitq_kv_dtype */
} bitq_kvdesc;

/* Bytes of the cache buffer.  Host only.  (A fresh cache needs no clearing.) */
bitq_status bitq_kv_cache_size(const bitq_kvdesc* kv, size_t* bytes);

/*
 * One scheduling step of a paged cache, on the GPU: from every request's
 * length before and after the step, pages are taken from a ring of free pages
 * for requests that grow and given back for requests that shrink (to 0: the
 * request is finished), and the new tokens get their slots.
 */
typedef struct {
    int32_t requests;      /* R, 1 .. 8192 */
    int32_t page;          /* tokens per page: a power of two, 8 .. 1024 */
    int32_t table_stride;  /* entries of one request's row of the table */
    int32_t ring;          /* entries of the ring = pages of the pool; ring * page < 2^31 */
    int32_t tokens;        /* T: most new tokens of a step, 1 .. 2^24 */
} bitq_kv_plan_desc;

/*
 * The plan buffer, written by bitq_kv_plan (i32 sections at multiples of 256
 * bytes, in this order):
 *   state [4]   head and count of the ring after the step (the next step's
 *               state_dev), new tokens n, requests refused
 *   len   [R]   lengths after the step
 *   start [R+1] start[r] .. start[r+1]-1 are request r's new tokens
 *   slot  [T]   slot of new token t in the pool (-1 from n on)
 *   req   [T]   its request (-1 from n on)
 *   pos   [T]   its position in the request (-1 from n on)
 */
bitq_status bitq_kv_plan_size(const bitq_kv_plan_desc* desc, size_t* bytes);

/*
 *   old_dev   i32 [R] lengths before the step: request r holds the pages
 *             table[r][0 .. ceil(old/page) - 1]
 *   new_dev   i32 [R] lengths asked for
 *   ring_dev  i32 [ring] page indices; `count` free ones from `head` on
 *             (wrapping round)
 *   state_dev i32 [2 or more] head, count; not inside plan_dev
 *   table_dev i32 [R][table_stride]
 *   plan_dev  bitq_kv_plan_size bytes, 256-byte aligned
 * Growing requests (new > old) are served in order of their index, each
 * taking its pages from the ring's head, as long as the pages and the T
 * tokens last; the first that does not fit, and every growing request after
 * it, is refused: its length and table stay, and it has no new tokens.
 * Shrinking requests (new < old) put the pages past ceil(new/page) at the
 * ring's end (their table entries stay and mean nothing any more).  A request
 * with old < 0, new < 0 or a length beyond table_stride * page is refused.
 * table_dev and ring_dev are updated in place; a repeated call on the same
 * arguments gives the same result.  count is taken as at most `ring`, and
 * what would not fit the ring is not put back.
 */
bitq_status bitq_kv_plan(const bitq_kv_plan_desc* desc, const int32_t* old_dev, const int32_t* new_dev,
                         int32_t* ring_dev, const int32_t* state_dev, int32_t* table_dev, void* plan_dev,
                         size_t plan_bytes, void* stream);

/*
 * Write the keys and values of `tokens` new tokens into their slots.
 *   k_dev, v_dev  [tokens][kv_heads][head_dim] in x_dtype (BITQ_DT_F32 or
 *                 BITQ_DT_BF16), token t starting k_stride (v_stride) elements
 *                 after token t-1 (at least kv_heads * head_dim); naturally
 *                 aligned (rows that are 16-byte aligned are read faster)
 *   slots_dev     i32 [tokens]; slots outside 0 .. pages*page-1 are skipped (the
 *                 rows of their tokens may be read all the same: k_dev and
 *                 v_dev hold all `tokens` rows); a slot given twice keeps
 *                 either token's values, element by element (int8: codes and
 *                 scale may be of different tokens)
 *   cache_dev     the cache, 256-byte aligned
 * bf16 caches round to nearest, ties to even; int8 caches quantize each row.
 * An int8 row with an infinity or NaN gets that as its scale and codes 0: every
 * value of it is NaN.
 * tokens = 0 does nothing; tokens <= 2^24, tokens * kv_heads <= 2^28.
 */
bitq_status bitq_kv_write(const bitq_kvdesc* kv, const void* k_dev, const void* v_dev, int32_t x_dtype,
                          int64_t k_stride, int64_t v_stride, const int32_t* slots_dev, int32_t tokens,
                          void* cache_dev, size_t cache_bytes, void* stream);

/*
 * Attention of one new token per request over the paged cache:
 *   out[r][a] = sum_t p_t V_t / sum_t p_t,  p_t = exp(scale q[r][a] . K_t)
 * over the tokens t of request r (its len_r tokens, or the last `window` of
 * them), query head a reading key-value head a / (heads / kv_heads).
 */
typedef struct {
    bitq_kvdesc kv;
    int32_t heads;         /* query heads, a multiple of kv_heads, <= 16384 */
    int32_t requests;      /* R, 1 .. 65535; requests * heads <= 2^23 */
    int32_t table_stride;  /* entries of one request's row of the table */
    int32_t max_len;       /* most tokens of a request, 1 .. table_stride * page */
    int32_t window;        /* 0: all tokens; else the last `window` tokens */
    int32_t q_dtype;       /* BITQ_DT_F32 or BITQ_DT_BF16 */
    int32_t out_dtype;     /* BITQ_DT_F32 or BITQ_DT_BF16 */
    float scale;           /* finite */
} bitq_attn_desc;

/*
 * Workspace of bitq_paged_attn: the partial results of requests whose tokens
 * are split over workgroups (0: none needed).  Its contents need no clearing
 * and carry nothing from call to call; calls that share it must be ordered.
 */
bitq_status bitq_paged_attn_workspace(const bitq_attn_desc* desc, size_t* bytes);

/*
 *   q_dev     [R][heads][head_dim] in q_dtype, request r starting q_stride
 *             elements after request r-1
 *   table_dev i32 [R][table_stride] page indices (an index outside the pool
 *             reads page 0)
 *   lens_dev  i32 [R] tokens of each request, the new one included; values
 *             below 0 count as 0, above max_len as max_len
 *   out_dev   [R][heads][head_dim] in out_dtype, contiguous
 *   lse_dev   f32 [R][heads] log(sum_t p_t), or NULL
 * A request without tokens gives out = 0 and lse = -inf.  Whatever the cache
 * holds outside a request's tokens, infinities and NaN included, has no
 * effect on its output.  NaN in its own q, keys or values gives NaN; so may an
 * infinity there.
 */
bitq_status bitq_paged_attn(const bitq_attn_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                            size_t cache_bytes, const int32_t* table_dev, const int32_t* lens_dev, void* out_dev,
                            float* lse_dev, void* ws_dev, size_t ws_bytes, void* stream);

/* ================================================ residual and norms */

/*
 * The residual update between two blocks, for rows of `width` elements:
 *   y  = post (.) u / sqrt(mean(u^2) + eps_post)   (y = u without post)
 *   r' = res_scale r + branch_scale gate (.) y     (no gate: 1; no r: 0)
 *   h  = pre (.) r' / sqrt(mean(r'^2) + eps_pre)   (h = r' without pre)
 * u is a block's output, r the residual stream, h the next block's input.
 * The norm of r' is taken from the unrounded r'.
 */
typedef struct {
    int32_t rows;          /* M, 1 .. 2^24 */
    int32_t width;         /* C, 1 .. 32768 */
    int32_t u_dtype;       /* BITQ_DT_F32 or BITQ_DT_BF16 */
    int32_t r_dtype;       /* of r and r' */
    int32_t w_dtype;       /* of post, gate and pre */
    int32_t out_dtype;     /* of h: BITQ_DT_F32, BITQ_DT_BF16 or BITQ_DT_ROW8 */
    int64_t u_stride, r_stride, ro_stride, h_stride;  /* elements between rows, >= width */
    int64_t gate_stride;   /* 0: one gate row for all rows; else >= width */
    float res_scale, branch_scale, eps_post, eps_pre; /* finite, eps >= 0 */
} bitq_norm_desc;

/* h in int8 rows: codes int8 [M] rows and one fp32 scale per row (the
 * arithmetic of bitq_quantize_act), what bitq_gemm_w8a8 takes.  A row with an
 * infinity or NaN gets that as its scale and codes 0: every value of it is NaN. */
#define BITQ_DT_ROW8 16

/*
 *   u_dev    [M][C]; r_dev [M][C] or NULL; post_dev [C] or NULL; gate_dev
 *            [C] or [M][C] or NULL; pre_dev [C] or NULL
 *   ro_dev   r' [M][C] in r_dtype, or NULL; may be r_dev itself
 *   h_dev    h [M][C] in out_dtype
 *   d_dev    f32 [M], the rows' scales (BITQ_DT_ROW8; else NULL)
 * All naturally aligned.  ro_dev and h_dev may not overlap any other buffer
 * of the call (but ro_dev = r_dev with equal strides).
 */
bitq_status bitq_block_norm(const bitq_norm_desc* desc, const void* u_dev, const void* r_dev, const void* post_dev,
                            const void* gate_dev, const void* pre_dev, void* ro_dev, void* h_dev, float* d_dev,
                            void* stream);

/* ================================================ int8 matrix product */

/*
 * y[m][n] = a_scale[m] w_scale[n] sum_k a[m][k] w[n][k], int8 rows with a
 * scale per token and per output channel.  The sum is exact (int32).
 */
typedef struct {
    int32_t M;        /* tokens, 1 .. 2^24 */
    int32_t N;        /* output channels, 1 .. 2^24; M * N <= 2^36 */
    int32_t K;        /* inputs, a multiple of 16, 16 .. 131056 */
    int32_t y_dtype;  /* BITQ_DT_F32 or BITQ_DT_BF16; BITQ_DT_F32 with BITQ_F_ACC_INT32 */
    int64_t lda, ldw; /* bytes between rows, multiples of 16, >= K, < 2^23 */
    int64_t ldy;      /* elements between rows, >= N */
    uint32_t flags;   /* 0, or BITQ_F_ACC_INT32: y receives the int32 sums */
} bitq_w8a8_desc;

/* Workspace of bitq_gemm_w8a8: the partial sums of calls whose k range is
 * split over workgroups (0: none needed).  Its contents need no clearing and
 * carry nothing from call to call; calls that share it must be ordered. */
bitq_status bitq_w8a8_workspace(const bitq_w8a8_desc* desc, size_t* bytes);

/*
 *   a_dev  int8 [M] rows, 16-byte aligned (e.g. the q section of a
 *          bitq_quantize_act buffer with lda = Kp and its d section as scales,
 *          or the rows of bitq_block_norm)
 *   w_dev  int8 [N] rows, 16-byte aligned
 *   a_scale_dev f32 [M], w_scale_dev f32 [N] (ignored, and may be NULL, with
 *          BITQ_F_ACC_INT32)
 *   y_dev  [M] rows in y_dtype, naturally aligned
 */
bitq_status bitq_gemm_w8a8(const bitq_w8a8_desc* desc, const void* a_dev, const float* a_scale_dev, const void* w_dev,
                           const float* w_scale_dev, void* y_dev, void* ws_dev, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITQ_LM_H */
