// Attention of several query rows: launches of bitq_prompt_attn and
// bitq_shared_attn, and the kernel that joins what they split.
#include "bitq_rows.h"

namespace bitq {

// Joins a row's partial results: NW waves to a row, each with a share of its
// pieces, 64 at a time: lane p has m and l of piece p, the accumulators are added
// with the weights 2^(m - M), AHEAD pieces' loads on their way together.  Bound by
// latency; one wave a row where there are many rows (4096 rows of 17 pieces, 36
// MB, 10 us), 16 where there are few (rows of 256, 14 of 187 pieces: 29 us with
// one).
template <int NE, int NW>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void rows_join_kernel(RowsArgs a, int Dp) {
    constexpr int AHEAD = 32 / NE;
    __shared__ float s_acc[NW][64 * NE], s_m[NW], s_l[NW];
    const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
    const uint32_t row = NW == 1 ? blockIdx.x * 4u + static_cast<uint32_t>(wave) : blockIdx.x;
    if (row >= static_cast<uint32_t>(a.T) * a.A) return;
    const int t = row / static_cast<uint32_t>(a.A);
    int p0 = 0;
    if (a.groups == 0) {
        if (t < rows_start(a, 0) || t >= rows_start(a, a.R)) return;  // (no request's row)
    } else {
        const int g = wave_search(a.groups, t, [&](int i) { return rows_start(a, i); });
        if (g < 0 || t >= rows_start(a, g + 1)) p0 = a.pieces;  // (in no group: its own tokens alone)
    }
    float acc[NE] = {}, M = -FLT_MAX, L = 0.0f;
    const int per = (a.all - p0 + NW - 1) / NW, end = NW == 1 ? a.all : min(a.all, p0 + (wave + 1) * per);
    for (int c = p0 + (NW == 1 ? 0 : wave * per); c < end; c += 64) {
        const int n = min(64, end - c);
        const float2 ml = a.ml[static_cast<size_t>(row) * a.all + c + min(lane, n - 1)];
        const bool has = lane < n && ml.y != 0.0f;  // (an l of NaN counts)
        float mn = has ? ml.x : -FLT_MAX;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor(mn, o, 64));
        mn = fmaxf(M, mn);
        const float f = __builtin_amdgcn_exp2f(M - mn), w = has ? __builtin_amdgcn_exp2f(ml.x - mn) : 0.0f;
        M = mn;
        float sum = has ? ml.y * w : 0.0f;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
        L = L * f + sum;
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] *= f;
        const uint64_t some = __ballot(has);
        const float* base = a.part + (static_cast<size_t>(row) * a.all + c) * Dp;
        for (int p = 0; p < n; p += AHEAD) {
            float v[AHEAD][NE];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
#pragma unroll
                for (int e = 0; e < NE; ++e) v[q][e] = base[min(p + q, n - 1) * Dp + min(lane + 64 * e, Dp - 1)];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const bool use = p + q < n && (some >> min(p + q, 63) & 1);  // (a piece without tokens has written no accumulator)
                const float wq = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), min(p + q, 63)));
#pragma unroll
                for (int e = 0; e < NE; ++e) acc[e] += use ? v[q][e] * wq : 0.0f;
            }
        }
    }
    if constexpr (NW > 1) {
        if (lane == 0) {
            s_m[wave] = M;
            s_l[wave] = L;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) s_acc[wave][lane + 64 * e] = acc[e];
        __syncthreads();
        if (wave != 0) return;
        M = s_m[0];
#pragma unroll
        for (int v = 1; v < NW; ++v) M = fmaxf(M, s_m[v]);
        L = 0.0f;
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
            const float f = __builtin_amdgcn_exp2f(s_m[v] - M);
            L += f * s_l[v];
#pragma unroll
            for (int e = 0; e < NE; ++e) acc[e] += f * s_acc[v][lane + 64 * e];
        }
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int d = lane + 64 * e;
        if (d < a.D) rows_store(a, static_cast<size_t>(row) * a.D + d, L == 0.0f ? 0.0f : acc[e] / L);
    }
    if (lane == 0 && a.lse) a.lse[row] = rows_lse(M, L);
}

static RowsArgs rows_args(const bitq_kvdesc& kv, const RowsPlan& plan, const RowsCall& c, int heads, int q_dtype, int out_dtype,
                          float scale) {
    const KvLayout L = kv_layout(kv);
    RowsArgs a{};
    a.q = c.q;
    a.cache = static_cast<const uint8_t*>(c.cache);
    a.table = c.table, a.start = c.start, a.lens = c.lens, a.prefix = c.prefix;
    a.out = c.out;
    a.lse = c.lse;
    a.ml = static_cast<float2*>(c.ws);
    a.part = plan.all ? reinterpret_cast<float*>(static_cast<uint8_t*>(c.ws) + plan.off_part) : nullptr;
    a.q_stride = c.q_stride;
    a.off_v = L.off_v, a.off_ks = L.off_ks, a.off_vs = L.off_vs;
    a.H = kv.kv_heads, a.A = heads, a.G = plan.group, a.D = kv.head_dim;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(kv.page));
    a.pages = kv.pages;
    a.all = plan.all;
    // (a scale of 0 weighs all tokens alike: so does one so small that no score counts)
    const float s = scale * 1.44269504088896340736f, mag = s < 0 ? -s : s;
    a.c = mag < FLT_MIN ? FLT_MIN : mag;
    a.negative = s < 0;
    a.odt = out_dtype;
    const int per16 = q_dtype == BITQ_DT_F32 ? 4 : 8;
    a.qvec = a.D % 8 == 0 && c.q_stride % per16 == 0 && aligned(c.q, 16);
    a.ovec = a.D % 8 == 0 && aligned(c.out, 16);
    return a;
}

static void launch_main(const bitq_kvdesc& kv, const RowsArgs& a, int rw, bool q32, void* stream) {
    const unsigned grid = (static_cast<unsigned>(a.tiles) * a.pieces + static_cast<unsigned>(a.own_tiles) * a.own_pieces) * a.H;
    if (kv.dtype == BITQ_KV_BF16) launch_rows_bf16(a, (a.D + 31) / 32, q32, rw, grid, stream);
    else launch_rows_int8(a, (a.D + 31) / 32, q32, rw, grid, stream);
}

template <int NE>
static void launch_rows_join(const RowsArgs& a, int Dp, hipStream_t st) {
    const unsigned rows = static_cast<unsigned>(a.T) * a.A;
    if (rows <= 1024 && a.all > 8) hipLaunchKernelGGL((rows_join_kernel<NE, 16>), dim3(rows), dim3(1024), 0, st, a, Dp);
    else hipLaunchKernelGGL((rows_join_kernel<NE, 1>), dim3((rows + 3) / 4), dim3(256), 0, st, a, Dp);
}
static void launch_rows_join(const RowsArgs& a, int Dp, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (Dp <= 64) launch_rows_join<1>(a, Dp, st);
    else if (Dp <= 128) launch_rows_join<2>(a, Dp, st);
    else launch_rows_join<4>(a, Dp, st);
}

int launch_prompt_attn(const bitq_prompt_desc& d, const RowsPlan& plan, const RowsCall& c, void* stream) {
    RowsArgs a = rows_args(d.kv, plan, c, d.heads, d.q_dtype, d.out_dtype, d.scale);
    a.R = d.requests, a.T = d.tokens;
    a.table_stride = d.table_stride, a.max_len = d.max_len, a.window = d.window, a.sinks = d.window ? d.sinks : 0;
    a.tiles = plan.main.tiles, a.pieces = plan.main.pieces;
    launch_main(d.kv, a, plan.main.rw, d.q_dtype == BITQ_DT_F32, stream);
    if (plan.all) launch_rows_join(a, plan.Dp, stream);
    return static_cast<int>(hipGetLastError());
}

int launch_shared_attn(const bitq_shared_desc& s, const RowsPlan& plan, const RowsCall& c, void* stream) {
    const bitq_attn_desc& d = s.attn;
    RowsArgs a = rows_args(d.kv, plan, c, d.heads, d.q_dtype, d.out_dtype, d.scale);
    const bool q32 = d.q_dtype == BITQ_DT_F32;
    a.R = a.T = d.requests, a.groups = s.groups, a.max_prefix = s.max_prefix;
    a.table_stride = d.table_stride, a.max_len = d.max_len;
    a.tiles = plan.main.tiles, a.pieces = plan.main.pieces;
    a.own_tiles = plan.own.tiles, a.own_pieces = plan.own.pieces, a.tps = plan.own.tiles / d.requests;
    if (plan.main.rw == plan.own.rw) {
        launch_main(d.kv, a, plan.main.rw, q32, stream);
    } else {
        a.own_tiles = 0;
        launch_main(d.kv, a, plan.main.rw, q32, stream);
        a.tiles = 0;
        a.own_tiles = plan.own.tiles;
        launch_main(d.kv, a, plan.own.rw, q32, stream);
    }
    launch_rows_join(a, plan.Dp, stream);
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
