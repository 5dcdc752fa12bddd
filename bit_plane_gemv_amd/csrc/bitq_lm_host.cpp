// Host side of the operators of bitq_lm.h: argument validation, launch plans
// and the C ABI entry points.
#include <algorithm>
#include <cmath>

#include "bitq_internal.h"

namespace bitq {
namespace {

size_t dtype_align(int32_t t) { return t == BITQ_DT_F32 ? 4 : t == BITQ_DT_BF16 ? 2 : 1; }
bool pow2(int32_t v) { return v > 0 && (v & (v - 1)) == 0; }

bitq_status check_page(int32_t page) {
    if (!pow2(page) || page < 8 || page > 1024)
        return fail(BITQ_E_SHAPE, "page=%d must be a power of two in [8, 1024]", page);
    return BITQ_OK;
}

bitq_status check_kv(const bitq_kvdesc& kv) {
    if (kv.dtype != BITQ_KV_BF16 && kv.dtype != BITQ_KV_INT8) return fail(BITQ_E_ARG, "unknown cache dtype %d", kv.dtype);
    if (kv.kv_heads < 1 || kv.kv_heads > 1024) return fail(BITQ_E_SHAPE, "kv_heads=%d out of range [1, 1024]", kv.kv_heads);
    if (kv.head_dim < 1 || kv.head_dim > 256) return fail(BITQ_E_SHAPE, "head_dim=%d out of range [1, 256]", kv.head_dim);
    if (bitq_status s = check_page(kv.page)) return s;
    if (kv.pages < 1 || static_cast<int64_t>(kv.pages) * kv.page > INT32_MAX)
        return fail(BITQ_E_SHAPE, "pages=%d: pages * page must be in [%d, 2^31)", kv.pages, kv.page);
    return BITQ_OK;
}

bitq_status check_plan(const bitq_kv_plan_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (d->requests < 1 || d->requests > 8192) return fail(BITQ_E_SHAPE, "requests=%d out of range [1, 8192]", d->requests);
    if (bitq_status s = check_page(d->page)) return s;
    if (d->table_stride < 1 || static_cast<int64_t>(d->table_stride) * d->page > INT32_MAX)
        return fail(BITQ_E_SHAPE, "table_stride=%d: table_stride * page must be in [%d, 2^31)", d->table_stride, d->page);
    if (d->ring < 1 || static_cast<int64_t>(d->ring) * d->page > INT32_MAX)
        return fail(BITQ_E_SHAPE, "ring=%d: ring * page must be in [%d, 2^31)", d->ring, d->page);
    if (d->tokens < 1 || d->tokens > (1 << 24)) return fail(BITQ_E_SHAPE, "tokens=%d out of range [1, 2^24]", d->tokens);
    return BITQ_OK;
}

bitq_status check_attn(const bitq_attn_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (bitq_status s = check_kv(d->kv)) return s;
    if (d->heads < 1 || d->heads > 16384 || d->heads % d->kv.kv_heads)
        return fail(BITQ_E_SHAPE, "heads=%d must be a multiple of kv_heads=%d, at most 16384", d->heads, d->kv.kv_heads);
    if (d->requests < 1 || d->requests > 65535) return fail(BITQ_E_SHAPE, "requests=%d out of range [1, 65535]", d->requests);
    if (static_cast<int64_t>(d->requests) * d->heads > (1 << 23))
        return fail(BITQ_E_SHAPE, "requests * heads is larger than 2^23");
    if (d->table_stride < 1) return fail(BITQ_E_SHAPE, "table_stride=%d must be positive", d->table_stride);
    if (d->max_len < 1 || d->max_len > static_cast<int64_t>(d->table_stride) * d->kv.page)
        return fail(BITQ_E_SHAPE, "max_len=%d out of range [1, table_stride * page]", d->max_len);
    if (d->max_len > INT32_MAX - 2 * kAttnUnit) return fail(BITQ_E_SHAPE, "max_len=%d is too long", d->max_len);
    if (d->window < 0) return fail(BITQ_E_SHAPE, "window=%d is negative", d->window);
    if ((d->q_dtype != BITQ_DT_F32 && d->q_dtype != BITQ_DT_BF16) ||
        (d->out_dtype != BITQ_DT_F32 && d->out_dtype != BITQ_DT_BF16))
        return fail(BITQ_E_ARG, "q_dtype and out_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (!std::isfinite(d->scale)) return fail(BITQ_E_ARG, "scale is not finite");
    return BITQ_OK;
}

bitq_status check_norm(const bitq_norm_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (d->rows < 1 || d->rows > (1 << 24)) return fail(BITQ_E_SHAPE, "rows=%d out of range [1, 2^24]", d->rows);
    if (d->width < 1 || d->width > 32768) return fail(BITQ_E_SHAPE, "width=%d out of range [1, 32768]", d->width);
    auto flt = [](int32_t t) { return t == BITQ_DT_F32 || t == BITQ_DT_BF16; };
    if (!flt(d->u_dtype) || !flt(d->r_dtype) || !flt(d->w_dtype))
        return fail(BITQ_E_ARG, "u_dtype, r_dtype and w_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (!flt(d->out_dtype) && d->out_dtype != BITQ_DT_ROW8)
        return fail(BITQ_E_ARG, "out_dtype must be BITQ_DT_F32, BITQ_DT_BF16 or BITQ_DT_ROW8");
    if (d->u_stride < d->width || d->r_stride < d->width || d->ro_stride < d->width || d->h_stride < d->width)
        return fail(BITQ_E_SHAPE, "a row stride is smaller than width=%d", d->width);
    if (d->gate_stride != 0 && d->gate_stride < d->width)
        return fail(BITQ_E_SHAPE, "gate_stride must be 0 or at least width=%d", d->width);
    const int64_t most = int64_t(1) << 40;  // row offsets stay far inside 64 bits
    if (d->u_stride > most || d->r_stride > most || d->ro_stride > most || d->h_stride > most || d->gate_stride > most)
        return fail(BITQ_E_SHAPE, "a row stride is larger than 2^40");
    if (!std::isfinite(d->res_scale) || !std::isfinite(d->branch_scale))
        return fail(BITQ_E_ARG, "res_scale and branch_scale must be finite");
    if (!(d->eps_post >= 0 && d->eps_pre >= 0) || !std::isfinite(d->eps_post) || !std::isfinite(d->eps_pre))
        return fail(BITQ_E_ARG, "eps_post and eps_pre must be finite and not negative");
    return BITQ_OK;
}

bitq_status check_w8a8(const bitq_w8a8_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (d->M < 1 || d->M > (1 << 24)) return fail(BITQ_E_SHAPE, "M=%d out of range [1, 2^24]", d->M);
    if (d->N < 1 || d->N > (1 << 24)) return fail(BITQ_E_SHAPE, "N=%d out of range [1, 2^24]", d->N);
    if (d->K < 16 || d->K > 131056 || d->K % 16)
        return fail(BITQ_E_SHAPE, "K=%d must be a multiple of 16 in [16, 131056]", d->K);
    for (const int64_t ld : {d->lda, d->ldw})
        if (ld < d->K || ld % 16 || ld >= (1 << 23))  // (256 rows stay within a 31-bit offset)
            return fail(BITQ_E_SHAPE, "lda and ldw must be multiples of 16 in [K, 2^23)");
    if (static_cast<int64_t>(d->M) * d->N > (int64_t(1) << 36))
        return fail(BITQ_E_SHAPE, "M * N = %lld is larger than 2^36", static_cast<long long>(d->M) * d->N);
    if (d->ldy < d->N || d->ldy > (int64_t(1) << 32)) return fail(BITQ_E_SHAPE, "ldy must be in [N, 2^32]");
    if (d->y_dtype != BITQ_DT_F32 && d->y_dtype != BITQ_DT_BF16)
        return fail(BITQ_E_ARG, "y_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (d->flags & ~BITQ_F_ACC_INT32) return fail(BITQ_E_ARG, "unknown flags 0x%x", d->flags);
    if ((d->flags & BITQ_F_ACC_INT32) && d->y_dtype != BITQ_DT_F32)
        return fail(BITQ_E_ARG, "BITQ_F_ACC_INT32 needs y_dtype = BITQ_DT_F32 (32-bit outputs)");
    return BITQ_OK;
}

bitq_status check_pages(const bitq_kv_pages_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (d->requests < 1 || d->requests > 8192) return fail(BITQ_E_SHAPE, "requests=%d out of range [1, 8192]", d->requests);
    if (bitq_status s = check_page(d->page)) return s;
    if (d->table_stride < 1 || static_cast<int64_t>(d->table_stride) * d->page > INT32_MAX)
        return fail(BITQ_E_SHAPE, "table_stride=%d: table_stride * page must be in [%d, 2^31)", d->table_stride, d->page);
    if (d->pool < 1 || static_cast<int64_t>(d->pool) * d->page > INT32_MAX)
        return fail(BITQ_E_SHAPE, "pool=%d: pool * page must be in [%d, 2^31)", d->pool, d->page);
    if (d->moves < 1 || d->moves > (1 << 28)) return fail(BITQ_E_SHAPE, "moves=%d out of range [1, 2^28]", d->moves);
    return BITQ_OK;
}

bitq_status check_rope(const bitq_rope_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    auto flt = [](int32_t t) { return t == BITQ_DT_F32 || t == BITQ_DT_BF16; };
    if (!flt(d->x_dtype) || !flt(d->out_dtype) || !flt(d->w_dtype))
        return fail(BITQ_E_ARG, "x_dtype, out_dtype and w_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (d->layout != BITQ_ROPE_HALF && d->layout != BITQ_ROPE_PAIRS) return fail(BITQ_E_ARG, "unknown layout %d", d->layout);
    if (d->tokens < 1 || d->tokens > (1 << 24)) return fail(BITQ_E_SHAPE, "tokens=%d out of range [1, 2^24]", d->tokens);
    if (d->q_heads < 0 || d->q_heads > 16384 || d->k_heads < 0 || d->k_heads > 16384 || d->q_heads + d->k_heads == 0)
        return fail(BITQ_E_SHAPE, "q_heads=%d and k_heads=%d must be in [0, 16384], one of them positive", d->q_heads, d->k_heads);
    if (static_cast<int64_t>(d->tokens) * (d->q_heads + d->k_heads) > (int64_t(1) << 28))
        return fail(BITQ_E_SHAPE, "tokens * (q_heads + k_heads) is larger than 2^28");
    if (d->head_dim < 1 || d->head_dim > 256) return fail(BITQ_E_SHAPE, "head_dim=%d out of range [1, 256]", d->head_dim);
    if (d->rot < 0 || d->rot > d->head_dim || d->rot % 2)
        return fail(BITQ_E_SHAPE, "rot=%d must be even, in [0, head_dim]", d->rot);
    if (!(d->eps >= 0) || !std::isfinite(d->eps) || !std::isfinite(d->mscale))
        return fail(BITQ_E_ARG, "eps and mscale must be finite, eps not negative");
    return BITQ_OK;
}

// (the factor of scores in powers of two)
bool scale_fits(float scale) { return std::isfinite(scale * 1.44269504088896340736f); }

bitq_status check_prompt(const bitq_prompt_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (bitq_status s = check_kv(d->kv)) return s;
    if (d->heads < 1 || d->heads > 16384 || d->heads % d->kv.kv_heads)
        return fail(BITQ_E_SHAPE, "heads=%d must be a multiple of kv_heads=%d, at most 16384", d->heads, d->kv.kv_heads);
    // (8192 requests x 1024 key-value heads, with a place for a tile each: a launch has fewer than 2^32 threads)
    if (d->requests < 1 || d->requests > 8192) return fail(BITQ_E_SHAPE, "requests=%d out of range [1, 8192]", d->requests);
    if (d->tokens < 1 || d->tokens > (1 << 20)) return fail(BITQ_E_SHAPE, "tokens=%d out of range [1, 2^20]", d->tokens);
    if (static_cast<int64_t>(d->tokens) * d->heads > (1 << 26)) return fail(BITQ_E_SHAPE, "tokens * heads is larger than 2^26");
    if (d->table_stride < 1) return fail(BITQ_E_SHAPE, "table_stride=%d must be positive", d->table_stride);
    if (d->max_len < 1 || d->max_len > static_cast<int64_t>(d->table_stride) * d->kv.page)
        return fail(BITQ_E_SHAPE, "max_len=%d out of range [1, table_stride * page]", d->max_len);
    if (d->max_len > INT32_MAX - 2 * kAttnUnit) return fail(BITQ_E_SHAPE, "max_len=%d is too long", d->max_len);
    if (d->window < 0) return fail(BITQ_E_SHAPE, "window=%d is negative", d->window);
    if (d->sinks < 0 || (d->sinks > 0 && d->window == 0))
        return fail(BITQ_E_SHAPE, "sinks=%d must be 0 without a window, and not negative", d->sinks);
    if ((d->q_dtype != BITQ_DT_F32 && d->q_dtype != BITQ_DT_BF16) ||
        (d->out_dtype != BITQ_DT_F32 && d->out_dtype != BITQ_DT_BF16))
        return fail(BITQ_E_ARG, "q_dtype and out_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (!scale_fits(d->scale)) return fail(BITQ_E_ARG, "scale * log2(e) is not finite");
    return BITQ_OK;
}

bitq_status check_shared(const bitq_shared_desc* d) {
    if (!d) return fail(BITQ_E_ARG, "desc is NULL");
    if (bitq_status s = check_attn(&d->attn)) return s;
    if (d->attn.requests > 8192) return fail(BITQ_E_SHAPE, "requests=%d out of range [1, 8192]", d->attn.requests);
    if (d->attn.window != 0) return fail(BITQ_E_SHAPE, "window=%d: a shared prefix is seen whole", d->attn.window);
    if (!scale_fits(d->attn.scale)) return fail(BITQ_E_ARG, "scale * log2(e) is not finite");
    if (d->groups < 1 || d->groups > d->attn.requests) return fail(BITQ_E_SHAPE, "groups=%d out of range [1, requests]", d->groups);
    if (d->max_prefix < 1 || d->max_prefix > d->attn.max_len)
        return fail(BITQ_E_SHAPE, "max_prefix=%d out of range [1, max_len]", d->max_prefix);
    return BITQ_OK;
}

// Whether [a, a + an) and [b, b + bn) have a byte in common.
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
    return p < q + bn && q < p + an;
}

struct Range {
    const void* at;
    size_t bytes;
    const char* name;
};
// Every output apart from every input and from the other outputs.
template <size_t NI, size_t NO>
bitq_status check_apart(const Range (&in)[NI], const Range (&out)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Range& r : in)
            if (overlap(out[i].at, out[i].bytes, r.at, r.bytes))
                return fail(BITQ_E_ARG, "%s may not overlap %s", out[i].name, r.name);
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes))
                return fail(BITQ_E_ARG, "%s may not overlap %s", out[i].name, out[j].name);
    }
    return BITQ_OK;
}

bitq_status check_pages_buffers(const KvPagesLayout& L, void* result, size_t result_bytes, void* ws, size_t ws_bytes) {
    if (!aligned(result, 256) || !aligned(ws, 256)) return fail(BITQ_E_ALIGN, "result_dev and ws_dev must be 256-byte aligned");
    if (result_bytes < L.total) return fail(BITQ_E_CAPACITY, "result buffer has %zu bytes, needs %zu", result_bytes, L.total);
    if (ws_bytes < L.ws_total) return fail(BITQ_E_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, L.ws_total);
    return BITQ_OK;
}

bitq_status check_rows_call(const bitq_kvdesc& kv, int heads, int64_t rows, int requests, int table_stride, int groups, int32_t q_dtype, int32_t out_dtype, const RowsCall& c,
                            size_t cache_bytes, const RowsPlan& plan, size_t ws_bytes) {
    if (!c.q || !c.cache || !c.table || !c.start || !c.lens || !c.out) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (c.q_stride < static_cast<int64_t>(heads) * kv.head_dim || c.q_stride > (int64_t(1) << 40))
        return fail(BITQ_E_SHAPE, "q_stride must be in [heads * head_dim, 2^40]");
    if (!aligned(c.q, dtype_align(q_dtype)) || !aligned(c.out, dtype_align(out_dtype)) || !aligned(c.table, 4) ||
        !aligned(c.start, 4) || !aligned(c.lens, 4) || !aligned(c.lse, 4))
        return fail(BITQ_E_ALIGN, "q_dev, out_dev, lse_dev, table_dev, start_dev and lens_dev must be naturally aligned");
    if (!aligned(c.cache, 256)) return fail(BITQ_E_ALIGN, "cache_dev must be 256-byte aligned");
    const size_t need = kv_layout(kv).total;
    if (cache_bytes < need) return fail(BITQ_E_CAPACITY, "cache has %zu bytes, needs %zu", cache_bytes, need);
    if (plan.ws_bytes > 0) {
        if (!c.ws) return fail(BITQ_E_ARG, "workspace is NULL");
        if (!aligned(c.ws, 256)) return fail(BITQ_E_ALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < plan.ws_bytes) return fail(BITQ_E_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, plan.ws_bytes);
    }
    const size_t row = static_cast<size_t>(heads) * kv.head_dim, r = 4 * static_cast<size_t>(requests), n = static_cast<size_t>(rows);
    const Range in[] = {{c.q, ((n - 1) * c.q_stride + row) * dtype_align(q_dtype), "q_dev"},
                        {c.cache, need, "cache_dev"},
                        {c.table, r * table_stride, "table_dev"},
                        {c.lens, r, "lens_dev"},
                        {c.start, 4 * (static_cast<size_t>(groups ? groups : requests) + 1), "start_dev"},
                        {c.prefix, 4 * static_cast<size_t>(groups), "prefix_dev"}};
    const Range out[] = {{c.out, n * row * dtype_align(out_dtype), "out_dev"},
                         {c.lse, c.lse ? n * heads * 4 : 0, "lse_dev"},
                         {plan.ws_bytes ? c.ws : nullptr, plan.ws_bytes, "workspace"}};
    return check_apart(in, out);
}

bitq_status check_device() {
    int is950 = 0;
    const int e = current_device_is_gfx950(&is950);
    if (e) return fail(BITQ_E_DEVICE, "HIP error %d while querying the device", e);
    if (!is950) return fail(BITQ_E_UNSUPPORTED, "current device is not gfx950");
    return BITQ_OK;
}

bitq_status launched(int e) {
    if (e) return fail(BITQ_E_DEVICE, "HIP launch error %d", e);
    return ok();
}

// Pieces for tiles of a call: enough workgroups to fill the GPU, each with two
// blocks or more (128 rows: one after the other; few rows: one for each wave).
int rows_pieces(int64_t tiles, int64_t span, int kv_heads, int groups_per_cu, int rw, int64_t most) {
    const int64_t want = 256 * groups_per_cu / std::max<int64_t>(1, tiles * kv_heads);
    const int64_t unit = rows_block(rw) * 2;
    return static_cast<int>(std::max<int64_t>(1, std::min(std::min<int64_t>(want, most), (span + unit - 1) / unit)));
}

void rows_workspace(RowsPlan& p, int64_t rows) {
    p.off_part = align256(static_cast<size_t>(rows) * p.all * 8);
    p.ws_bytes = p.off_part + static_cast<size_t>(rows) * p.all * p.Dp * 4;
}

}  // namespace

RowsPlan prompt_plan(const bitq_prompt_desc& d) {
    RowsPlan p{};
    p.Dp = static_cast<int>(round_up(d.kv.head_dim, 32));
    p.group = d.heads / d.kv.kv_heads;
    const int nc = p.Dp / 32;
    const bool q32 = d.q_dtype == BITQ_DT_F32;
    const int64_t rows = static_cast<int64_t>(d.tokens) * p.group;  // of a key-value head
    p.main.rw = rows <= 32 * static_cast<int64_t>(d.requests) ? 1 : 4;
    p.main.tiles = static_cast<int>(rows / (32 * p.main.rw) + d.requests);
    const int64_t span = d.window > 0 ? std::min<int64_t>(d.max_len, int64_t(d.window) + d.sinks + 32 * p.main.rw / p.group) : d.max_len;
    // (partial results of at most 256 MB)
    const int64_t cap = std::min<int64_t>(512, (int64_t(1) << 26) / (static_cast<int64_t>(d.tokens) * d.heads * (p.Dp + 2)));
    // (tiles in use: one for each request with tokens at least)
    p.main.pieces = rows_pieces(std::max<int64_t>(std::min(d.requests, d.tokens), (rows + 32 * p.main.rw - 1) / (32 * p.main.rw)), span, d.kv.kv_heads,
                                rows_groups_per_cu(d.kv.dtype, nc, q32, p.main.rw), p.main.rw, cap);
    if (p.main.pieces > 1) {
        p.all = p.main.pieces;
        rows_workspace(p, static_cast<int64_t>(d.tokens) * d.heads);
    }
    return p;
}

RowsPlan shared_plan(const bitq_shared_desc& s) {
    const bitq_attn_desc& d = s.attn;
    RowsPlan p{};
    p.Dp = static_cast<int>(round_up(d.kv.head_dim, 32));
    p.group = d.heads / d.kv.kv_heads;
    const int nc = p.Dp / 32, H = d.kv.kv_heads;
    const bool q32 = d.q_dtype == BITQ_DT_F32;
    const int64_t rows = static_cast<int64_t>(d.requests) * p.group;
    p.main.rw = rows <= 32 * static_cast<int64_t>(s.groups) ? 1 : 4;
    p.main.tiles = static_cast<int>(rows / (32 * p.main.rw) + s.groups);
    // One launch for both parts if both take few rows, so that each fills what the other leaves (40 requests in 5 groups, 32
    // heads of 64, int8: 54 -> 48 us); else a launch each (64 requests on 16384 tokens, with two
    // terms of p: 95 us, and 101 with own tokens on tiles of 128 rows).
    p.own.rw = p.group <= 32 ? 1 : 4;
    p.own.tiles = d.requests * ((p.group + 32 * p.own.rw - 1) / (32 * p.own.rw));
    // (partial results of at most 256 MB where there are few rows; a piece of the prefix and one of the own tokens always: 2^23
    // rows of 256 elements need 17 GB)
    const int64_t cap = std::max<int64_t>(1, std::min<int64_t>(512, (int64_t(1) << 25) / (static_cast<int64_t>(d.requests) * d.heads * (p.Dp + 2))));
    p.main.pieces = rows_pieces(std::max<int64_t>(s.groups, (rows + 32 * p.main.rw - 1) / (32 * p.main.rw)), s.max_prefix, H,
                                rows_groups_per_cu(d.kv.dtype, nc, q32, p.main.rw), p.main.rw, cap);
    p.own.pieces = rows_pieces(p.own.tiles, std::max(d.max_len - s.max_prefix, 1), H,
                               rows_groups_per_cu(d.kv.dtype, nc, q32, p.own.rw), p.own.rw, cap);
    p.all = p.main.pieces + p.own.pieces;
    rows_workspace(p, static_cast<int64_t>(d.requests) * d.heads);
    return p;
}

AttnPlan attn_plan(const bitq_attn_desc& d) {
    AttnPlan p{};
    p.Dp = static_cast<int>(round_up(d.kv.head_dim, 32));
    p.group = d.heads / d.kv.kv_heads;
    p.tiles = (p.group + 15) / 16;
    p.items = d.requests * d.kv.kv_heads * p.tiles;
    const int64_t span = d.window > 0 ? std::min<int64_t>(d.max_len, static_cast<int64_t>(d.window) + 31) : d.max_len;
    const int64_t units = (span + kAttnUnit - 1) / kAttnUnit;  // of the longest request
    const bool q32 = d.q_dtype == BITQ_DT_F32;
    // A workgroup for each item while the longest is short: the split's second
    // kernel costs about 4 us, a unit of an item 0.6 us and more with its row.
    // Where items fill half of the CUs and more the others' work hides it.
    // Measured, bf16, whole / split, us: 16 items with rows of 128, 512 tokens
    // 7.9 / 9.5, 1024 12.4 / 10.0; rows of 64, 1024 8.8 / 8.9; of 256, 256 tokens
    // 9.0 / 11.6, 512 13.3 / 11.9.  128 items, rows of 128, 1024 tokens 15.1 /
    // 17.8, 2048 31.5 / 31.7; of 256, 512 15.9 / 18.4, 1024 33 / 32.  2048 items
    // of up to 256 ragged tokens 30 / 41.
    const bool whole = units <= 8 && units * p.Dp <= (p.items >= 128 ? 1024 : 640);
    p.split = !whole && d.requests <= kAttnMaxSplitRequests && p.items * units < INT32_MAX;
    // (the CUs filled as often as registers allow; two units and more for a
    // workgroup measured slower: one request of 2049 tokens 17.5 against 15.1 us)
    const int64_t all = p.items * units, full = 256 * attn_groups_per_cu(d.kv.dtype, p.Dp / 32, q32);
    p.grid = p.split ? static_cast<int>(std::min(full, all)) : p.items;
    // Short spans of more items than workgroups fit at once: workgroups of one
    // wave, of which four times as many do.  Measured, 2048 items of up to 32 /
    // 64 / 128 tokens, bf16, us with 1 and 4 waves: rows of 128 8.6 and 12.8 /
    // 11.8 and 13.8 / 16.7 and 15.7; of 256 21 and 43 / 26 and 45 / 39 and 54;
    // 512 items with rows of 128 (all fit) 6.1 and 5.4 / 6.9 and 5.6.
    const bool one = !p.split && p.items > full && (span <= 64 || full == 256);
    p.waves = one ? 1 : kAttnWaves;
    if (p.split) {
        // prefix sums of the requests' units, then two partial results per workgroup: 16 heads x (Dp + 2) floats
        p.off_part = align256(4 * (static_cast<size_t>(d.requests) + 1));
        p.ws_bytes = p.off_part + static_cast<size_t>(p.grid) * 2 * 16 * (p.Dp + 2) * 4;
    }
    return p;
}

}  // namespace bitq

using namespace bitq;

extern "C" {

bitq_status bitq_kv_cache_size(const bitq_kvdesc* kv, size_t* bytes) {
    if (!kv || !bytes) return fail(BITQ_E_ARG, "kv/bytes is NULL");
    if (bitq_status s = check_kv(*kv)) return s;
    *bytes = kv_layout(*kv).total;
    return ok();
}

bitq_status bitq_kv_plan_size(const bitq_kv_plan_desc* desc, size_t* bytes) {
    if (bitq_status s = check_plan(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = kv_plan_layout(*desc).total;
    return ok();
}

bitq_status bitq_kv_plan(const bitq_kv_plan_desc* desc, const int32_t* old_dev, const int32_t* new_dev,
                         int32_t* ring_dev, const int32_t* state_dev, int32_t* table_dev, void* plan_dev,
                         size_t plan_bytes, void* stream) {
    if (bitq_status s = check_plan(desc)) return s;
    if (!old_dev || !new_dev || !ring_dev || !state_dev || !table_dev || !plan_dev)
        return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!aligned(old_dev, 4) || !aligned(new_dev, 4) || !aligned(ring_dev, 4) || !aligned(state_dev, 4) ||
        !aligned(table_dev, 4))
        return fail(BITQ_E_ALIGN, "old_dev, new_dev, ring_dev, state_dev and table_dev must be 4-byte aligned");
    if (!aligned(plan_dev, 256)) return fail(BITQ_E_ALIGN, "plan_dev must be 256-byte aligned");
    const size_t need = kv_plan_layout(*desc).total;
    if (plan_bytes < need) return fail(BITQ_E_CAPACITY, "plan buffer has %zu bytes, needs %zu", plan_bytes, need);
    // (every workgroup reads the state and the old lengths: they may not be
    // overwritten by another workgroup of the same launch)
    const char *p = static_cast<const char*>(plan_dev);
    for (const void* in : {static_cast<const void*>(state_dev), static_cast<const void*>(old_dev),
                           static_cast<const void*>(new_dev)}) {
        const char* c = static_cast<const char*>(in);
        const size_t bytes = in == state_dev ? 8 : 4 * static_cast<size_t>(desc->requests);
        if (c + bytes > p && c < p + need)
            return fail(BITQ_E_ARG, "old_dev, new_dev and state_dev may not lie in plan_dev (use two plan buffers in turn)");
    }
    if (bitq_status s = check_device()) return s;
    return launched(launch_kv_plan(*desc, old_dev, new_dev, ring_dev, state_dev, table_dev, plan_dev, stream));
}

bitq_status bitq_kv_pages_size(const bitq_kv_pages_desc* desc, size_t* bytes) {
    if (bitq_status s = check_pages(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = kv_pages_layout(*desc).total;
    return ok();
}

bitq_status bitq_kv_pages_workspace(const bitq_kv_pages_desc* desc, size_t* bytes) {
    if (bitq_status s = check_pages(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = kv_pages_layout(*desc).ws_total;
    return ok();
}

bitq_status bitq_kv_fork(const bitq_kv_pages_desc* desc, const int32_t* src_dev, const int32_t* keep_dev,
                         const int32_t* len_dev, int32_t* ring_dev, const int32_t* state_dev, const int32_t* table_dev,
                         int32_t* table_out_dev, void* result_dev, size_t result_bytes, void* ws_dev, size_t ws_bytes,
                         void* stream) {
    if (bitq_status s = check_pages(desc)) return s;
    if (desc->moves < desc->requests) return fail(BITQ_E_SHAPE, "moves=%d: a fork lists up to requests=%d copies", desc->moves, desc->requests);
    if (!src_dev || !keep_dev || !len_dev || !ring_dev || !state_dev || !table_dev || !table_out_dev || !result_dev || !ws_dev)
        return fail(BITQ_E_ARG, "a device pointer is NULL");
    for (const void* p : {static_cast<const void*>(src_dev), static_cast<const void*>(keep_dev), static_cast<const void*>(len_dev),
                          static_cast<const void*>(ring_dev), static_cast<const void*>(state_dev),
                          static_cast<const void*>(table_dev), static_cast<const void*>(table_out_dev)})
        if (!aligned(p, 4)) return fail(BITQ_E_ALIGN, "the int32 buffers must be 4-byte aligned");
    const KvPagesLayout L = kv_pages_layout(*desc);
    if (bitq_status s = check_pages_buffers(L, result_dev, result_bytes, ws_dev, ws_bytes)) return s;
    const size_t r = 4 * static_cast<size_t>(desc->requests), table = r * desc->table_stride;
    const Range in[] = {{src_dev, r, "src_dev"}, {keep_dev, r, "keep_dev"}, {len_dev, r, "len_dev"}, {state_dev, 8, "state_dev"},
                        {table_dev, table, "table_dev"}};
    const Range out[] = {{ring_dev, 4 * static_cast<size_t>(desc->pool), "ring_dev"}, {table_out_dev, table, "table_out_dev"},
                         {result_dev, L.total, "result_dev"}, {ws_dev, L.ws_total, "ws_dev"}};
    if (bitq_status s = check_apart(in, out)) return s;
    if (bitq_status s = check_device()) return s;
    return launched(launch_kv_fork(*desc, src_dev, keep_dev, len_dev, ring_dev, state_dev, table_dev, table_out_dev, result_dev,
                                   ws_dev, stream));
}

bitq_status bitq_kv_compact(const bitq_kv_pages_desc* desc, const int32_t* len_dev, const int32_t* table_dev,
                            int32_t* table_out_dev, int32_t* ring_dev, void* result_dev, size_t result_bytes,
                            void* ws_dev, size_t ws_bytes, void* stream) {
    if (bitq_status s = check_pages(desc)) return s;
    if (!len_dev || !table_dev || !table_out_dev || !ring_dev || !result_dev || !ws_dev)
        return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!aligned(len_dev, 4) || !aligned(table_dev, 4) || !aligned(table_out_dev, 4) || !aligned(ring_dev, 4))
        return fail(BITQ_E_ALIGN, "the int32 buffers must be 4-byte aligned");
    const KvPagesLayout L = kv_pages_layout(*desc);
    if (bitq_status s = check_pages_buffers(L, result_dev, result_bytes, ws_dev, ws_bytes)) return s;
    const size_t r = 4 * static_cast<size_t>(desc->requests), table = r * desc->table_stride;
    const Range in[] = {{len_dev, r, "len_dev"}, {table_dev, table, "table_dev"}};
    const Range out[] = {{ring_dev, 4 * static_cast<size_t>(desc->pool), "ring_dev"}, {table_out_dev, table, "table_out_dev"},
                         {result_dev, L.total, "result_dev"}, {ws_dev, L.ws_total, "ws_dev"}};
    if (bitq_status s = check_apart(in, out)) return s;
    if (bitq_status s = check_device()) return s;
    return launched(launch_kv_compact(*desc, len_dev, table_dev, table_out_dev, ring_dev, result_dev, ws_dev, stream));
}

bitq_status bitq_kv_copy(const bitq_kvdesc* kv, const int32_t* frm_dev, const int32_t* to_dev, int32_t moves,
                         void* cache_dev, size_t cache_bytes, void* stream) {
    if (!kv) return fail(BITQ_E_ARG, "kv is NULL");
    if (bitq_status s = check_kv(*kv)) return s;
    if (moves < 0 || moves > (1 << 28)) return fail(BITQ_E_SHAPE, "moves=%d out of range [0, 2^28]", moves);
    if (!cache_dev) return fail(BITQ_E_ARG, "cache_dev is NULL");
    if (moves > 0 && (!frm_dev || !to_dev)) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!aligned(frm_dev, 4) || !aligned(to_dev, 4)) return fail(BITQ_E_ALIGN, "frm_dev and to_dev must be 4-byte aligned");
    if (!aligned(cache_dev, 256)) return fail(BITQ_E_ALIGN, "cache_dev must be 256-byte aligned");
    const size_t need = kv_layout(*kv).total;
    if (cache_bytes < need) return fail(BITQ_E_CAPACITY, "cache has %zu bytes, needs %zu", cache_bytes, need);
    const size_t list = 4 * static_cast<size_t>(moves);
    if (overlap(frm_dev, list, cache_dev, need) || overlap(to_dev, list, cache_dev, need))
        return fail(BITQ_E_ARG, "frm_dev and to_dev may not lie in the cache");
    if (bitq_status s = check_device()) return s;
    if (moves == 0) return ok();
    return launched(launch_kv_copy(*kv, frm_dev, to_dev, moves, cache_dev, stream));
}

bitq_status bitq_rope_table(const bitq_rope_freq* f, uint64_t* table) {
    if (!f || !table) return fail(BITQ_E_ARG, "freq/table is NULL");
    if (f->rot < 2 || f->rot > 256 || f->rot % 2) return fail(BITQ_E_SHAPE, "rot=%d must be even, in [2, 256]", f->rot);
    if (f->kind < BITQ_ROPE_PLAIN || f->kind > BITQ_ROPE_BAND) return fail(BITQ_E_ARG, "unknown kind %d", f->kind);
    if (!(f->base > 1) || !std::isfinite(f->base)) return fail(BITQ_E_ARG, "base must be finite and larger than 1");
    if (f->kind != BITQ_ROPE_PLAIN && (!(f->factor > 0) || !std::isfinite(f->factor)))
        return fail(BITQ_E_ARG, "factor must be finite and positive");
    const bool parts = f->kind == BITQ_ROPE_RAMP || f->kind == BITQ_ROPE_BAND;
    if (parts && (!(f->trained > 0) || !std::isfinite(f->trained) || !(f->turns_scale > 0) || !(f->turns_keep > f->turns_scale) ||
                  !std::isfinite(f->turns_keep)))
        return fail(BITQ_E_ARG, "trained, turns_scale and turns_keep must be finite, positive, and turns_keep > turns_scale");
    const long double tau = 6.283185307179586476925286766559005768L;
    const int rot = f->rot;
    // where a pair makes x turns over the trained positions (a number of a pair)
    auto at = [&](long double x) { return rot * std::log(f->trained / (x * tau)) / (2 * std::log(static_cast<long double>(f->base))); };
    long double lo = 0, hi = 1;
    if (f->kind == BITQ_ROPE_RAMP) {
        lo = std::max(std::floor(at(f->turns_keep)), 0.0L);
        hi = std::min(std::ceil(at(f->turns_scale)), static_cast<long double>(rot - 1));
    }
    for (int i = 0; i < rot / 2; ++i) {
        const long double w = std::pow(static_cast<long double>(f->base), -2.0L * i / rot);
        long double keep = 1;  // how much of the plain frequency stays
        if (f->kind == BITQ_ROPE_LINEAR) keep = 0;
        if (f->kind == BITQ_ROPE_RAMP) keep = 1 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001L), 0.0L), 1.0L);
        if (f->kind == BITQ_ROPE_BAND) {
            const long double t = (f->trained * w / tau - f->turns_scale) / (f->turns_keep - f->turns_scale);
            keep = std::min(std::max(t, 0.0L), 1.0L);
        }
        long double turns = (w * keep + (keep < 1 ? w / f->factor * (1 - keep) : 0)) / tau;
        turns -= std::floor(turns);
        const long double fixed = std::floor(turns * 18446744073709551616.0L + 0.5L);  // 2^64
        table[i] = fixed >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(fixed);
    }
    return ok();
}

bitq_status bitq_qk_rope(const bitq_rope_desc* desc, const void* q_dev, int64_t q_stride, const void* k_dev,
                         int64_t k_stride, const void* qw_dev, const void* kw_dev, const uint64_t* table_dev,
                         const int32_t* pos_dev, void* qo_dev, int64_t qo_stride, void* ko_dev, int64_t ko_stride,
                         void* stream) {
    if (bitq_status s = check_rope(desc)) return s;
    const bitq_rope_desc& d = *desc;
    if (!pos_dev || (d.q_heads && (!q_dev || !qo_dev)) || (d.k_heads && (!k_dev || !ko_dev)) || (d.rot && !table_dev))
        return fail(BITQ_E_ARG, "a device pointer is NULL");
    const size_t ax = dtype_align(d.x_dtype), ao = dtype_align(d.out_dtype), aw = dtype_align(d.w_dtype);
    const RopeRows r[4] = {{q_dev, d.q_heads, q_stride}, {k_dev, d.k_heads, k_stride}, {qo_dev, d.q_heads, qo_stride},
                           {ko_dev, d.k_heads, ko_stride}};
    static const char* const names[4] = {"q_stride", "k_stride", "qo_stride", "ko_stride"};
    for (int i = 0; i < 4; ++i)  // (row offsets of 2^24 tokens stay inside 63 bits)
        if (r[i].heads && (r[i].stride < static_cast<int64_t>(r[i].heads) * d.head_dim || r[i].stride > (int64_t(1) << 36)))
            return fail(BITQ_E_SHAPE, "%s must be in [heads * head_dim, 2^36]", names[i]);
    if (!aligned(q_dev, ax) || !aligned(k_dev, ax) || !aligned(qo_dev, ao) || !aligned(ko_dev, ao) || !aligned(qw_dev, aw) ||
        !aligned(kw_dev, aw) || !aligned(table_dev, 8) || !aligned(pos_dev, 4))
        return fail(BITQ_E_ALIGN, "every buffer must be naturally aligned");
    // Rows of q and k may lie side by side in one buffer (a projection's): equal strides show them apart token by token.
    auto span = [&](const RopeRows& x, size_t size) {
        return x.heads ? (static_cast<size_t>(d.tokens - 1) * x.stride + static_cast<size_t>(x.heads) * d.head_dim) * size : 0;
    };
    auto clash = [&](const RopeRows& x, size_t xs, const RopeRows& y, size_t ys) {
        if (!x.heads || !y.heads || !overlap(x.at, span(x, xs), y.at, span(y, ys))) return false;
        const int64_t row = x.stride * static_cast<int64_t>(xs);
        if (row != y.stride * static_cast<int64_t>(ys)) return true;
        const int64_t gap = static_cast<int64_t>(reinterpret_cast<intptr_t>(y.at) - reinterpret_cast<intptr_t>(x.at)) % row;
        const int64_t at = gap < 0 ? gap + row : gap;  // where y's rows begin in x's
        return at < static_cast<int64_t>(x.heads) * d.head_dim * static_cast<int64_t>(xs) ||
               at + static_cast<int64_t>(y.heads) * d.head_dim * static_cast<int64_t>(ys) > row;
    };
    bool bad = clash(r[2], ao, r[3], ao);
    for (int i = 0; i < 2; ++i)
        for (int j = 2; j < 4; ++j) {
            const bool place = j == i + 2 && r[i].at == r[j].at && r[i].stride == r[j].stride && d.x_dtype == d.out_dtype;
            bad = bad || (!place && clash(r[i], ax, r[j], ao));
        }
    const Range rest[] = {{qw_dev, qw_dev ? aw * d.head_dim : 0, ""}, {kw_dev, kw_dev ? aw * d.head_dim : 0, ""},
                          {table_dev, table_dev ? 4 * static_cast<size_t>(d.rot) : 0, ""},
                          {pos_dev, 4 * static_cast<size_t>(d.tokens), ""}};
    for (const Range& x : rest)
        for (int j = 2; j < 4; ++j) bad = bad || (x.bytes && r[j].heads && overlap(x.at, x.bytes, r[j].at, span(r[j], ao)));
    if (bad) return fail(BITQ_E_ARG, "qo_dev and ko_dev may be q_dev and k_dev with the same type and stride, and overlap nothing else");
    if (bitq_status s = check_device()) return s;
    return launched(launch_qk_rope(d, r, qw_dev, kw_dev, table_dev, pos_dev, stream));
}

bitq_status bitq_kv_write(const bitq_kvdesc* kv, const void* k_dev, const void* v_dev, int32_t x_dtype,
                          int64_t k_stride, int64_t v_stride, const int32_t* slots_dev, int32_t tokens,
                          void* cache_dev, size_t cache_bytes, void* stream) {
    if (!kv) return fail(BITQ_E_ARG, "kv is NULL");
    if (bitq_status s = check_kv(*kv)) return s;
    if (x_dtype != BITQ_DT_F32 && x_dtype != BITQ_DT_BF16)
        return fail(BITQ_E_ARG, "x_dtype must be BITQ_DT_F32 or BITQ_DT_BF16");
    if (tokens < 0 || tokens > (1 << 24)) return fail(BITQ_E_SHAPE, "tokens=%d out of range [0, 2^24]", tokens);
    if (static_cast<int64_t>(tokens) * kv->kv_heads > (int64_t(1) << 28))
        return fail(BITQ_E_SHAPE, "tokens * kv_heads is larger than 2^28");
    const int64_t row = static_cast<int64_t>(kv->kv_heads) * kv->head_dim;
    for (const int64_t st : {k_stride, v_stride})
        if (st < row || st > (int64_t(1) << 40))
            return fail(BITQ_E_SHAPE, "k_stride and v_stride must be in [kv_heads * head_dim, 2^40]");
    if (!cache_dev) return fail(BITQ_E_ARG, "cache_dev is NULL");
    if (tokens > 0 && (!k_dev || !v_dev || !slots_dev)) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!aligned(k_dev, dtype_align(x_dtype)) || !aligned(v_dev, dtype_align(x_dtype)) || !aligned(slots_dev, 4))
        return fail(BITQ_E_ALIGN, "k_dev, v_dev and slots_dev must be naturally aligned");
    if (!aligned(cache_dev, 256)) return fail(BITQ_E_ALIGN, "cache_dev must be 256-byte aligned");
    const size_t need = kv_layout(*kv).total;
    if (cache_bytes < need) return fail(BITQ_E_CAPACITY, "cache has %zu bytes, needs %zu", cache_bytes, need);
    if (bitq_status s = check_device()) return s;
    if (tokens == 0) return ok();
    return launched(launch_kv_write(*kv, k_dev, v_dev, x_dtype, k_stride, v_stride, slots_dev, tokens, cache_dev, stream));
}

bitq_status bitq_paged_attn_workspace(const bitq_attn_desc* desc, size_t* bytes) {
    if (bitq_status s = check_attn(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = attn_plan(*desc).ws_bytes;
    return ok();
}

bitq_status bitq_paged_attn(const bitq_attn_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                            size_t cache_bytes, const int32_t* table_dev, const int32_t* lens_dev, void* out_dev,
                            float* lse_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    if (bitq_status s = check_attn(desc)) return s;
    if (!q_dev || !cache_dev || !table_dev || !lens_dev || !out_dev) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (q_stride < static_cast<int64_t>(desc->heads) * desc->kv.head_dim || q_stride > (int64_t(1) << 40))
        return fail(BITQ_E_SHAPE, "q_stride must be in [heads * head_dim, 2^40]");
    if (!aligned(q_dev, dtype_align(desc->q_dtype)) || !aligned(out_dev, dtype_align(desc->out_dtype)) ||
        !aligned(table_dev, 4) || !aligned(lens_dev, 4) || !aligned(lse_dev, 4))
        return fail(BITQ_E_ALIGN, "q_dev, out_dev, lse_dev, table_dev and lens_dev must be naturally aligned");
    if (!aligned(cache_dev, 256)) return fail(BITQ_E_ALIGN, "cache_dev must be 256-byte aligned");
    const size_t need = kv_layout(desc->kv).total;
    if (cache_bytes < need) return fail(BITQ_E_CAPACITY, "cache has %zu bytes, needs %zu", cache_bytes, need);
    const AttnPlan plan = attn_plan(*desc);
    if (plan.ws_bytes > 0) {
        if (!ws_dev) return fail(BITQ_E_ARG, "workspace is NULL");
        if (!aligned(ws_dev, 256)) return fail(BITQ_E_ALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < plan.ws_bytes)
            return fail(BITQ_E_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, plan.ws_bytes);
    }
    if (bitq_status s = check_device()) return s;
    return launched(launch_paged_attn(*desc, plan, q_dev, q_stride, cache_dev, table_dev, lens_dev, out_dev, lse_dev,
                                      ws_dev, stream));
}

bitq_status bitq_prompt_attn_workspace(const bitq_prompt_desc* desc, size_t* bytes) {
    if (bitq_status s = check_prompt(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = prompt_plan(*desc).ws_bytes;
    return ok();
}

bitq_status bitq_shared_attn_workspace(const bitq_shared_desc* desc, size_t* bytes) {
    if (bitq_status s = check_shared(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = shared_plan(*desc).ws_bytes;
    return ok();
}

bitq_status bitq_prompt_attn(const bitq_prompt_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                             size_t cache_bytes, const int32_t* table_dev, const int32_t* start_dev,
                             const int32_t* lens_dev, void* out_dev, float* lse_dev, void* ws_dev, size_t ws_bytes,
                             void* stream) {
    if (bitq_status s = check_prompt(desc)) return s;
    const RowsCall c{q_dev, q_stride, cache_dev, table_dev, start_dev, lens_dev, nullptr, out_dev, lse_dev, ws_dev};
    const RowsPlan plan = prompt_plan(*desc);
    if (bitq_status s = check_rows_call(desc->kv, desc->heads, desc->tokens, desc->requests, desc->table_stride, 0, desc->q_dtype, desc->out_dtype, c,
                                        cache_bytes, plan, ws_bytes))
        return s;
    if (bitq_status s = check_device()) return s;
    return launched(launch_prompt_attn(*desc, plan, c, stream));
}

bitq_status bitq_shared_attn(const bitq_shared_desc* desc, const void* q_dev, int64_t q_stride, const void* cache_dev,
                             size_t cache_bytes, const int32_t* table_dev, const int32_t* lens_dev,
                             const int32_t* start_dev, const int32_t* prefix_dev, void* out_dev, float* lse_dev,
                             void* ws_dev, size_t ws_bytes, void* stream) {
    if (bitq_status s = check_shared(desc)) return s;
    if (!prefix_dev) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!aligned(prefix_dev, 4)) return fail(BITQ_E_ALIGN, "prefix_dev must be 4-byte aligned");
    const RowsCall c{q_dev, q_stride, cache_dev, table_dev, start_dev, lens_dev, prefix_dev, out_dev, lse_dev, ws_dev};
    const RowsPlan plan = shared_plan(*desc);
    const bitq_attn_desc& d = desc->attn;
    if (bitq_status s = check_rows_call(d.kv, d.heads, d.requests, d.requests, d.table_stride, desc->groups, d.q_dtype, d.out_dtype, c, cache_bytes,
                                        plan, ws_bytes))
        return s;
    if (bitq_status s = check_device()) return s;
    return launched(launch_shared_attn(*desc, plan, c, stream));
}

bitq_status bitq_block_norm(const bitq_norm_desc* desc, const void* u_dev, const void* r_dev, const void* post_dev,
                            const void* gate_dev, const void* pre_dev, void* ro_dev, void* h_dev, float* d_dev,
                            void* stream) {
    if (bitq_status s = check_norm(desc)) return s;
    if (!u_dev || !h_dev) return fail(BITQ_E_ARG, "u_dev/h_dev is NULL");
    const bool row8 = desc->out_dtype == BITQ_DT_ROW8;
    if (row8 && !d_dev) return fail(BITQ_E_ARG, "BITQ_DT_ROW8 needs d_dev");
    if (!row8 && d_dev) return fail(BITQ_E_ARG, "d_dev belongs to BITQ_DT_ROW8");
    if (ro_dev == r_dev && ro_dev && desc->ro_stride != desc->r_stride)
        return fail(BITQ_E_SHAPE, "ro_dev = r_dev needs equal strides");
    if (h_dev == u_dev || h_dev == r_dev || h_dev == ro_dev || (ro_dev && ro_dev == u_dev))
        return fail(BITQ_E_ARG, "h_dev and ro_dev may not be another buffer of the call (but ro_dev = r_dev)");
    if (!aligned(u_dev, dtype_align(desc->u_dtype)) || !aligned(r_dev, dtype_align(desc->r_dtype)) ||
        !aligned(ro_dev, dtype_align(desc->r_dtype)) || !aligned(post_dev, dtype_align(desc->w_dtype)) ||
        !aligned(gate_dev, dtype_align(desc->w_dtype)) || !aligned(pre_dev, dtype_align(desc->w_dtype)) ||
        !aligned(h_dev, dtype_align(desc->out_dtype)) || !aligned(d_dev, 4))
        return fail(BITQ_E_ALIGN, "every buffer must be naturally aligned");
    if (bitq_status s = check_device()) return s;
    return launched(launch_block_norm(*desc, u_dev, r_dev, post_dev, gate_dev, pre_dev, ro_dev, h_dev, d_dev, stream));
}

bitq_status bitq_w8a8_workspace(const bitq_w8a8_desc* desc, size_t* bytes) {
    if (bitq_status s = check_w8a8(desc)) return s;
    if (!bytes) return fail(BITQ_E_ARG, "bytes is NULL");
    *bytes = w8a8_plan(*desc).ws_bytes;
    return ok();
}

bitq_status bitq_gemm_w8a8(const bitq_w8a8_desc* desc, const void* a_dev, const float* a_scale_dev, const void* w_dev,
                           const float* w_scale_dev, void* y_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    if (bitq_status s = check_w8a8(desc)) return s;
    if (!a_dev || !w_dev || !y_dev) return fail(BITQ_E_ARG, "a device pointer is NULL");
    if (!(desc->flags & BITQ_F_ACC_INT32) && (!a_scale_dev || !w_scale_dev))
        return fail(BITQ_E_ARG, "a scale pointer is NULL");
    if (!aligned(a_dev, 16) || !aligned(w_dev, 16)) return fail(BITQ_E_ALIGN, "a_dev and w_dev must be 16-byte aligned");
    if (!aligned(a_scale_dev, 4) || !aligned(w_scale_dev, 4) || !aligned(y_dev, dtype_align(desc->y_dtype)))
        return fail(BITQ_E_ALIGN, "the scales and y_dev must be naturally aligned");
    const W8A8Plan plan = w8a8_plan(*desc);
    if (plan.ws_bytes > 0) {
        if (!ws_dev) return fail(BITQ_E_ARG, "workspace is NULL");
        if (!aligned(ws_dev, 256)) return fail(BITQ_E_ALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < plan.ws_bytes)
            return fail(BITQ_E_CAPACITY, "workspace has %zu bytes, needs %zu", ws_bytes, plan.ws_bytes);
    }
    if (bitq_status s = check_device()) return s;
    return launched(launch_gemm_w8a8(*desc, plan, a_dev, a_scale_dev, w_dev, w_scale_dev, y_dev, ws_dev, stream));
}

}  // extern "C"
