/*
 * bitq_lm.h -- the operators that stand between the packed linear layers of a
 * decoder: a paged key-value cache (page tables and slot maps built on the
 * GPU, cache writes, attention of one new token per request, of several, and
 * of requests that share a prefix; requests forked and pages compacted), the
 * norms and rotation of queries and keys, the residual update of a block with
 * its norms, and the int8 matrix product for layers kept in 8 bits.
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

/* ================================== attention of several query rows */

/*
 * Attention of the new tokens of each request, one or many, over the paged
 * cache (which holds them already):
 *   out[i][a] = sum_t p_t V_t / sum_t p_t,  p_t = exp(scale q[i][a] . K_t)
 * Request r's new tokens are rows start[r] .. start[r+1]-1 of q, the last
 * n = start[r+1] - start[r] of its lens[r] tokens; row start[r] + j stands at
 * position x = lens[r] - n + j and sees the tokens t <= x of its request: all of
 * them, or with a window those with t > x - window and the first `sinks`
 * tokens, which stay visible.  Query head a reads key-value head
 * a / (heads / kv_heads).
 */
typedef struct {
    bitq_kvdesc kv;
    int32_t heads;         /* query heads, a multiple of kv_heads, <= 16384 */
    int32_t requests;      /* R, 1 .. 8192 */
    int32_t tokens;        /* T: rows of q, 1 .. 2^20; tokens * heads <= 2^26 */
    int32_t table_stride;  /* entries of one request's row of the table */
    int32_t max_len;       /* most tokens of a request, 1 .. table_stride * page */
    int32_t window;        /* 0: all tokens; else the last `window` tokens */
    int32_t sinks;         /* first tokens that stay visible; 0 without a window */
    int32_t q_dtype;       /* BITQ_DT_F32 or BITQ_DT_BF16 */
    int32_t out_dtype;     /* BITQ_DT_F32 or BITQ_DT_BF16 */
    float scale;           /* scale log2(e) finite */
} bitq_prompt_desc;

/* Workspace of bitq_prompt_attn: partial results where tokens are split over
 * workgroups (0: none needed).  Its contents need no clearing and carry
 * nothing from call to call; calls that share it must be ordered. */
bitq_status bitq_prompt_attn_workspace(const bitq_prompt_desc* desc, size_t* bytes);

/*
 *   q_dev     [T][heads][head_dim] in q_dtype, row i starting q_stride elements
 *             after row i-1
 *   table_dev i32 [R][table_stride] page indices (an index outside the pool
 *             reads page 0)
 *   start_dev i32 [R+1], ascending (bitq_kv_plan's start); values are taken as
 *             at least 0 and at most T, a request whose end lies before its
 *             start has no rows.  (Where they do not ascend, the results are
 *             undefined; no access leaves the buffers.)
 *   lens_dev  i32 [R] tokens of each request, its new ones included (0 ..
 *             max_len, others count as the nearer end); rows that would stand
 *             before position 0 see nothing
 *   out_dev   [T][heads][head_dim] in out_dtype, contiguous
 *   lse_dev   f32 [T][heads] log(sum_t p_t), or NULL
 * A row that sees no token gives out = 0 and lse = -inf; rows outside
 * start[0] .. start[R]-1 are left as they were.  out_dev, lse_dev and ws_dev
 * may not overlap another buffer of the call.  Whatever the cache holds in
 * places that a row does not see, infinities and NaN included, has no effect
 * on it.  NaN in its own q or in keys or values that it sees gives NaN; so may
 * an infinity there.  Scores are held as fp32 numbers, in powers of two: one for
 * which scale log2(e) q . K is beyond fp32 counts as an infinity.  So are weights
 * times values before the division by their sum: tokens that a row sees, times
 * the largest of their values, up to 2^119.
 */
bitq_status bitq_prompt_attn(const bitq_prompt_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                             size_t cache_bytes, const int32_t* table_dev, const int32_t* start_dev,
                             const int32_t* lens_dev, void* out_dev, float* lse_dev, void* ws_dev, size_t ws_bytes,
                             void* stream);

/*
 * bitq_paged_attn for requests of which groups begin with the same tokens: the
 * keys and values of such a prefix are read once for its group instead of once
 * for each request.  Requests start[g] .. start[g+1]-1 are group g, and their
 * first prefix[g] tokens are those of its first request, whose pages are read
 * (pages may be common to the group's tables, as bitq_kv_fork leaves them, or
 * copies).  Requests in no group have no prefix.
 */
typedef struct {
    bitq_attn_desc attn;   /* window = 0; requests <= 8192; scale log2(e) finite */
    int32_t groups;        /* 1 .. requests */
    int32_t max_prefix;    /* most tokens of a prefix, 1 .. attn.max_len */
} bitq_shared_desc;

/* As bitq_prompt_attn's, but never 0: each row has a partial result of the prefix
 * and one of its own tokens at least, requests * heads * 2 * (4 Dp + 8) bytes. */
bitq_status bitq_shared_attn_workspace(const bitq_shared_desc* desc, size_t* bytes);

/*
 * Buffers as for bitq_paged_attn, and
 *   start_dev  i32 [groups+1], ascending, values taken as at least 0 and at
 *              most R; a group whose end lies before its start has no requests
 *              (where they do not ascend, as for bitq_prompt_attn)
 *   prefix_dev i32 [groups], 0 .. max_prefix (others count as the nearer end)
 * A request shorter than its group's prefix sees its own length of it.
 * Scores and values as for bitq_prompt_attn.
 */
bitq_status bitq_shared_attn(const bitq_shared_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                             size_t cache_bytes, const int32_t* table_dev, const int32_t* lens_dev,
                             const int32_t* start_dev, const int32_t* prefix_dev, void* out_dev, float* lse_dev,
                             void* ws_dev, size_t ws_bytes, void* stream);

/* ============================================== pages of the cache */

/*
 * Requests forked, cut and freed, and the pool compacted.  Both calls find out
 * from the tables and lengths alone which pages are held, so pages may be held
 * by any number of requests (as bitq_kv_fork leaves them) and bitq_kv_plan can
 * take further ones at any time.  bitq_kv_plan gives back the pages of a
 * request that shrinks whoever else holds them: while pages are shared,
 * requests are cut and freed by bitq_kv_fork.
 */
typedef struct {
    int32_t requests;      /* R, 1 .. 8192 */
    int32_t page;          /* tokens per page: a power of two, 8 .. 1024 */
    int32_t table_stride;  /* entries of one request's row of the table; table_stride * page < 2^31 */
    int32_t pool;          /* pages of the pool = entries of the ring; pool * page < 2^31 */
    int32_t moves;         /* M: places of the list of page copies, 1 .. 2^28 (bitq_kv_fork: at least R) */
} bitq_kv_pages_desc;

/*
 * The result buffer of both calls (i32 sections at multiples of 256 bytes, in
 * this order):
 *   state [4]  head and count of the ring after the call, page copies n, and
 *              (fork) requests that did not get what they asked for / (compact)
 *              pages below which every held page now lies
 *   len   [R]  lengths after the call
 *   frm   [M]  page copies to make in the cache of every layer, frm[i] to
 *   to    [M]  to[i], i < n (-1 from n on): what bitq_kv_copy takes
 */
bitq_status bitq_kv_pages_size(const bitq_kv_pages_desc* desc, size_t* bytes);
bitq_status bitq_kv_pages_workspace(const bitq_kv_pages_desc* desc, size_t* bytes);  /* needs no clearing */

/*
 * Request r becomes the first keep[r] tokens of request src[r] as it was before
 * the call: src = r, keep = len leaves it; src = r, keep < len cuts it (0: frees
 * it); another src forks from that request (the steps of a beam search, more
 * samples of one prompt).  Whole pages are shared.  A page that a request ends
 * inside is its own afterwards, so that new tokens can follow: it stays with
 * the request that had it or else with the first that asks for it, and the
 * others get copies of it in pages from the ring (also the first, if another
 * request holds that page as a whole one).  Pages that nobody holds any more go
 * to the ring's end, in order of their index.
 *   src_dev, keep_dev, len_dev  i32 [R]; len outside 0 .. table_stride * page
 *                counts as the nearer end
 *   ring_dev     i32 [pool], state_dev i32 [2 or more] head, count: as for
 *                bitq_kv_plan; ring_dev is updated in place
 *   table_dev    i32 [R][table_stride]; table_out_dev the same, receives the
 *                tables after the call (entries past a request's pages are left
 *                as they were)
 *   result_dev   bitq_kv_pages_size bytes, ws_dev bitq_kv_pages_workspace
 *                bytes, both 256-byte aligned
 * src outside 0 .. R-1, or keep outside 0 .. len[src]: the request stays as it
 * was.  Copies are granted in order of the requests' index; one that the ring
 * has no page for ends at its last whole page instead (its len says so).
 * Both count in state[3].  Page indices outside the pool are handed on and
 * otherwise ignored.  A repeated call on the same arguments gives the same result.
 * The outputs may not overlap the inputs or each other (but ring_dev).
 */
bitq_status bitq_kv_fork(const bitq_kv_pages_desc* desc, const int32_t* src_dev, const int32_t* keep_dev,
                         const int32_t* len_dev, int32_t* ring_dev, const int32_t* state_dev, const int32_t* table_dev,
                         int32_t* table_out_dev, void* result_dev, size_t result_bytes, void* ws_dev, size_t ws_bytes,
                         void* stream);

/*
 * Moves held pages to the pool's low end: the highest held page to the lowest
 * free place, the next to the next, while that lies below it and the M places
 * of the list last.  With M >= pool the held pages are then 0 .. n-1 (and the
 * pool's upper part can be used otherwise).
 *   len_dev, table_dev, table_out_dev, result_dev, ws_dev  as for bitq_kv_fork
 *   ring_dev  i32 [pool]: receives the pages that no request holds, in order, from
 *             place 0 (entries past them are left as they were)
 */
bitq_status bitq_kv_compact(const bitq_kv_pages_desc* desc, const int32_t* len_dev, const int32_t* table_dev,
                            int32_t* table_out_dev, int32_t* ring_dev, void* result_dev, size_t result_bytes,
                            void* ws_dev, size_t ws_bytes, void* stream);

/*
 * Copies pages of one layer's cache (keys, values and scales): page frm[i] to
 * page to[i], i < moves.  Pairs with an index outside the pool are skipped.
 * No page may be copied to twice in a call, or be both copied from and to.
 *   frm_dev, to_dev i32 [moves]; cache_dev 256-byte aligned
 * moves = 0 does nothing.
 */
bitq_status bitq_kv_copy(const bitq_kvdesc* kv, const int32_t* frm_dev, const int32_t* to_dev, int32_t moves,
                         void* cache_dev, size_t cache_bytes, void* stream);

/* ================================= queries and keys: norms and positions */

typedef enum {
    BITQ_ROPE_HALF = 0,   /* pairs (x[i], x[i + rot/2]) */
    BITQ_ROPE_PAIRS = 1   /* pairs (x[2i], x[2i + 1]) */
} bitq_rope_layout;

/*
 * Frequencies of the rotation: pair i turns by f_i radians per position,
 * f_i = base^(-2i/rot), stretched for contexts longer than the trained ones by
 * dividing by `factor`
 *   BITQ_ROPE_PLAIN   none
 *   BITQ_ROPE_LINEAR  all of them
 *   BITQ_ROPE_RAMP    by the pairs' numbers: d(x) = rot ln(trained / (2 pi x)) /
 *                     (2 ln base) is where a pair makes x turns over the trained
 *                     positions; t = clamp((i - lo) / (hi - lo), 0, 1) with lo =
 *                     max(floor(d(turns_keep)), 0), hi = min(ceil(d(turns_scale)),
 *                     rot - 1) (hi - lo at least 0.001): f (1 - t) + f / factor t
 *   BITQ_ROPE_BAND    by the turns themselves: t = clamp((trained f / (2 pi) -
 *                     turns_scale) / (turns_keep - turns_scale), 0, 1):
 *                     f t + f / factor (1 - t)
 */
typedef enum { BITQ_ROPE_PLAIN = 0, BITQ_ROPE_LINEAR = 1, BITQ_ROPE_RAMP = 2, BITQ_ROPE_BAND = 3 } bitq_rope_kind;
typedef struct {
    int32_t rot;           /* elements of a head that are rotated: even, 2 .. 256 */
    int32_t kind;          /* bitq_rope_kind */
    double base;           /* > 1 */
    double factor;         /* > 0; not for BITQ_ROPE_PLAIN */
    double trained;        /* > 0, turns_keep > turns_scale > 0; BITQ_ROPE_RAMP and _BAND */
    double turns_keep, turns_scale;
} bitq_rope_freq;

/*
 * Host only.  table receives rot/2 entries: the fraction of a turn per position
 * as a 64-bit fixed-point number, f_i / (2 pi) 2^64 mod 2^64 rounded (computed
 * with 64 bits: off by less than 1/2 + 12 f_i / (2 pi) units; a program with
 * frequencies of its own fills the table in itself).  bitq_qk_rope cuts position
 * times entry to 32 bits of a turn: for frequencies up to 1, angles are off by
 * less than 2^-30 turns at every position below 2^31.
 */
bitq_status bitq_rope_table(const bitq_rope_freq* freq, uint64_t* table);

/*
 * Queries and keys of new tokens, head by head:
 *   x' = w (.) x / sqrt(mean(x^2) + eps)   (x' = x without w)
 * (squares and their sum in fp32: elements up to 2^59, and with eps = 0 a
 * largest one of 2^-40 or more)
 * and the first rot elements of x' rotated, each pair (u, v) by its angle
 * a = position * f_i:
 *   (mscale (u cos a - v sin a), mscale (v cos a + u sin a))
 */
typedef struct {
    int32_t tokens;        /* T, 1 .. 2^24; tokens * (q_heads + k_heads) <= 2^28 */
    int32_t q_heads, k_heads;  /* 0 .. 16384, not both 0 */
    int32_t head_dim;      /* 1 .. 256 */
    int32_t rot;           /* even, 0 .. head_dim (0: norms only) */
    int32_t layout;        /* bitq_rope_layout */
    int32_t x_dtype;       /* of q and k: BITQ_DT_F32 or BITQ_DT_BF16 */
    int32_t out_dtype;     /* of the outputs */
    int32_t w_dtype;       /* of the norms' weights */
    float eps, mscale;     /* finite, eps >= 0 */
} bitq_rope_desc;

/*
 *   q_dev [T][q_heads][head_dim], k_dev [T][k_heads][head_dim] in x_dtype
 *         (NULL with no heads), token t starting q_stride (k_stride) elements
 *         after token t-1 (at least heads * head_dim)
 *   qw_dev, kw_dev [head_dim] in w_dtype, or NULL: no norm
 *   table_dev u64 [rot/2] (bitq_rope_table; NULL with rot = 0), 8-byte aligned
 *   pos_dev   i32 [T] positions (bitq_kv_plan's pos); the rows of a token with
 *             a negative one are left as they were
 *   qo_dev, ko_dev  outputs in out_dtype, with strides of their own; may be q_dev,
 *             k_dev themselves with the same type and stride, and overlap
 *             nothing else of the call
 * All naturally aligned (16-byte aligned rows and parts of 8 elements are
 * read faster).
 */
bitq_status bitq_qk_rope(const bitq_rope_desc* desc, const void* q_dev, int64_t q_stride, const void* k_dev,
                         int64_t k_stride, const void* qw_dev, const void* kw_dev, const uint64_t* table_dev,
                         const int32_t* pos_dev, void* qo_dev, int64_t qo_stride, void* ko_dev, int64_t ko_stride,
                         void* stream);

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
