// Host side of the operators of bitq_lm.h: argument validation, launch plans
// and the C ABI entry points.
#include <algorithm>
#include <cmath>

#include "bitq_internal.h"

namespace bitq {
namespace {

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

size_t dtype_align(int32_t t) { return t == BITQ_DT_F32 ? 4 : t == BITQ_DT_BF16 ? 2 : 1; }

}  // namespace

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
