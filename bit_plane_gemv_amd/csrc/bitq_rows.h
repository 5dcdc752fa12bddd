// Attention of several query rows over the paged cache of libbitq: the kernel
// of bitq_prompt_attn and bitq_shared_attn, compiled per cache type in
// bitq_rows_bf16.hip and bitq_rows_int8.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>

#include "bitq_device.h"

namespace bitq {

// out = sum_t p_t V_t / sum_t p_t, p_t = exp(scale q . K_t), for rows (new token
// x query head) that read the same key-value head of one request.  Keys and
// values are read once for a tile of 32 or 128 rows.  One pass over the tokens:
// running maximum m, sum l and accumulator O per row, all fp32.
//
// Matrix cores.  v_mfma_f32_32x32x16_bf16 takes the products transposed,
//   S[32 tokens][32 rows] = K q^T,   O^T[Dp][32 rows] += V^T P:
// lane l = 32 h + j holds 8 consecutive k of row (column) j of A (B), and rows
// 8 b + 4 h + i (b, i < 4) of column j of D.  Row 8 b + 4 h + i of a score tile is
// given token 16 (b / 2) + 8 h + 4 (b % 2) + i, so the 16 scores of a lane are the
// 2 x 8 consecutive tokens that the B operands of the second product need from
// that lane: nothing moves between lanes, and a row's statistics lie in one
// column (two lanes).  V's layout (8 tokens of an element together) makes its
// A operand one 16-byte read.
//
// Tokens come in blocks that are copied straight from the cache into LDS, two
// stages of them, one in flight while the other is worked on.  Copies move
// groups of 8 tokens (a page has whole groups), so a page's index is the same
// for a whole copy instruction.  Keys are stored with their 16-byte pieces
// exchanged within a row by the row's number, so that the reads of a score tile
// (one piece of 32 rows) fall on all banks alike.
//   RW = 4: 128 rows, 32 to each of the 4 waves, which share blocks of 64 tokens.
//   RW = 1: 32 rows; each wave takes every W-th block of 32 tokens for itself
//           (no meeting of the waves until the end), and the waves' results are
//           joined in LDS.  For few rows, where the memory is the bound.
// A tile's tokens may be split over `pieces` workgroups; rows_join_kernel joins.
//
// Precision.  Cache rows are exact in bf16; int8 scales are applied in fp32, to
// the scores and to p.  fp32 q is split into 3 bf16 terms, which hold its 24
// bits.  p is split into 3 terms for fp32 outputs and into 2 for bf16 ones: 2
// terms err by 2^-17 of each weight, 2^-8 of the output's own rounding, and cost
// a quarter of the matrix work less.  One term would err by as much as that
// rounding and make the kernel no faster than the softmax's own instructions
// allow.  m follows the maximum only when it has grown by more than 2^8, which
// changes no result (p may then be up to 2^8).
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

enum RowsMode { kRowsPrompt = 0, kRowsPrefix = 1, kRowsOwn = 2 };

struct RowsArgs {
    const void* q;
    const uint8_t* cache;
    const int32_t *table, *start, *lens, *prefix;
    void* out;
    float* lse;
    float* part;           // [T A][all pieces][Dp], not normalised
    float2* ml;            // [T A][all pieces]: m (in powers of two), l
    int64_t q_stride;
    size_t off_v, off_ks, off_vs;
    int mode, R, T;        // segments (requests or groups) and rows of q
    int H, A, G, D, page_shift, pages, table_stride, max_len, window, sinks, max_prefix;
    int tiles;             // places for tiles (an upper bound of the tiles)
    int tps, groups;       // kRowsOwn: tiles per segment; groups
    int pieces, piece0, all;  // pieces a tile is split into, the first one's place, and the places of a row; all = 0: no split
    float c;               // |scale| log2(e) (> 0); a negative scale turns q's sign
    bool negative, q32, qvec, ovec;  // q32: fp32 q
    int odt;
};

template <int KVT, int NC, bool F32, int RW>
struct RowsShape {
    static constexpr bool I8 = KVT == BITQ_KV_INT8;
    static constexpr int Dp = 32 * NC, ES = I8 ? 1 : 2;
    static constexpr int W = rows_waves(NC, RW);
    static constexpr int BT = rows_block(RW);  // tokens of a block
    static constexpr int ROWS = 32 * RW;
    static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
    static constexpr int KB = BT * Dp * ES, STAGE = 2 * KB + (I8 ? 8 * BT : 0);
    static constexpr int TEAMS = RW == 4 ? 1 : W;
    static constexpr int GROUPS = BT / 8 / (RW == 4 ? W : 1);  // groups of 8 tokens that a wave copies
    static constexpr int GB = 8 * Dp * ES, IPG = (GB + 1023) / 1024;
    static constexpr int COPIES = GROUPS * (2 * IPG + (I8 ? 2 : 0));
    static constexpr int CN = Dp * ES / 16;                   // 16-byte pieces of a key
    static constexpr int ORow = Dp + 4;                       // floats of a row when the waves' results meet
    static constexpr int JOIN = RW == 4 ? 0 : W * 32 * (ORow + 2) * 4;
    static constexpr int LDS = rows_lds(KVT, NC, RW);
    static_assert(LDS >= TEAMS * 2 * STAGE && LDS >= JOIN, "stages, then the waves' results");
    // piece c of row r is stored at piece c ^ swizzle(r); rows 8 further on differ in ODD of a piece's offset
    static constexpr __device__ __forceinline__ int swizzle(int r) {
        return CN % 8 == 0 ? (r & 3) | ((r >> 3) & 1) << 2 : CN % 4 == 0 ? ((r >> 1) & 1) | ((r >> 3) & 1) << 1 : (r >> 3) & 1;
    }
    static constexpr uint32_t ODD = CN % 8 == 0 ? 64 : CN % 4 == 0 ? 32 : 16;
};

// A value of a table that no kernel of this launch writes, at a place that is
// the same for the whole wave: through the scalar cache.
__device__ __forceinline__ int scalar_i32(const int32_t* p, size_t i) {
    return *(reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p)) + i);
}

template <int N>
__device__ __forceinline__ void rows_wait_copies() {
    static_assert(N < 64, "vmcnt is a 6-bit count");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));  // vmcnt(N)
    asm volatile("" ::: "memory");
}
// this wave's LDS reads are done
__device__ __forceinline__ void rows_wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (7 << 4));  // lgkmcnt(0)
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void copy_lds4(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, static_cast<int>(voff), 0, 0, 0);
#endif
}

// 8 int8 codes as bf16 (exact)
__device__ __forceinline__ bf16x8_t rows_codes(uint32_t lo, uint32_t hi) {
    bf16x8_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(lo >> (8 * e))));
        v[4 + e] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(hi >> (8 * e))));
    }
    return v;
}

// x = sum of the N bf16 terms, each the rounding of what the ones before leave
template <int N>
__device__ __forceinline__ void rows_terms(const float* x, bf16x8_t (&t)[N]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[n][e] = static_cast<__bf16>(r[e]);
            if (n + 1 < N) r[e] -= static_cast<float>(t[n][e]);
        }
}

// of the two lanes 32 h + j of a column
__device__ __forceinline__ float pair_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// ---------------------------------------------------- segments and their rows
__device__ __forceinline__ int rows_start(const RowsArgs& a, int i) { return min(max(a.start[i], 0), a.T); }
__device__ __forceinline__ int rows_len(const RowsArgs& a, int i) { return min(max(a.lens[i], 0), a.max_len); }

// Largest i in [0, n) with key(i) <= x (key ascending; -1: none), by the whole
// wave: 64 keys at a time.  n <= 64^3.
template <class F>
__device__ __forceinline__ int wave_search(int n, int x, F key) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int step = n > 4096 ? 4096 : n > 64 ? 64 : 1; step; step /= 64) {
        const int i = base + lane * step;
        const bool in = i < n && key(min(i, n - 1)) <= x;
        const int c = __builtin_popcountll(__ballot(in));
        if (c == 0) return -1;
        base += (c - 1) * step;
    }
    return base;
}

// The prefix of group g as all of its rows use it: its first request holds it.
__device__ __forceinline__ int group_prefix(const RowsArgs& a, int g, int first) {
    return min(min(max(a.prefix[g], 0), a.max_prefix), rows_len(a, first));
}

__device__ __forceinline__ void rows_store(const RowsArgs& a, size_t i, float v) {
    if (a.odt == BITQ_DT_F32) static_cast<float*>(a.out)[i] = v;
    else static_cast<uint16_t*>(a.out)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ uint32_t rows_pair(float x, float y) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)) |
           (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(y))) << 16);
}
// elements d .. d + 3 of an output row (i: element 0 of the row)
__device__ __forceinline__ void rows_store4(const RowsArgs& a, size_t i, int d, f32x4_t v) {
    if (a.ovec) {  // (D a multiple of 8)
        if (d >= a.D) return;
        if (a.odt == BITQ_DT_F32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + i + d) = v;
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + i + d) = make_uint2(rows_pair(v[0], v[1]), rows_pair(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < a.D) rows_store(a, i + d + e, v[e]);
    }
}
__device__ __forceinline__ float rows_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

template <int KVT, int NC, bool F32, int RW>
__global__ __launch_bounds__(64 * rows_waves(NC, RW), rows_groups_per_cu(KVT, NC, F32, RW)) void rows_attn_kernel(RowsArgs a) {
    using Z = RowsShape<KVT, NC, F32, RW>;
    constexpr bool I8 = Z::I8;
    constexpr int Dp = Z::Dp, ES = Z::ES, W = Z::W, BT = Z::BT, NQ = Z::NQ, NP = Z::NP, CN = Z::CN, T16 = BT / 16;
    __shared__ __align__(16) uint8_t s_mem[Z::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6), h = lane >> 5, j = lane & 31;

    // ---- the tile: heads fastest (an XCD, blockIdx % 8, then sees few heads and
    // shares their keys in its L2), last tiles first (a prompt's longest)
    const uint32_t id = blockIdx.x, rest = id / static_cast<uint32_t>(a.H);
    const int hk = id - rest * a.H, slot = a.tiles - 1 - static_cast<int>(rest / static_cast<uint32_t>(a.pieces));
    const int piece = rest % static_cast<uint32_t>(a.pieces);
    int seg, tile, s0, n;  // segment, tile of it, its first row token and their number
    if (a.mode == kRowsOwn) {
        seg = slot / a.tps;
        tile = slot - seg * a.tps;
        s0 = seg;
        n = 1;
    } else {
        // the tiles of segment r lie from floor(start[r] G / ROWS) + r on: ceil(n G / ROWS) of them always fit
        auto key = [&](int r) { return rows_start(a, r) * a.G / Z::ROWS + r; };
        seg = wave_search(a.R, slot, key);
        if (seg < 0) return;
        seg = wave_uniform(seg);
        s0 = wave_uniform(rows_start(a, seg));
        n = wave_uniform(rows_start(a, seg + 1)) - s0;
        tile = slot - (s0 * a.G / Z::ROWS + seg);
        if (n <= 0 || tile * Z::ROWS >= n * a.G) return;
    }
    const int rows = n * a.G, x0 = tile * Z::ROWS;
    const int xw = x0 + (RW == 4 ? 32 * wave : 0), mine = min(32, rows - xw);  // this wave's rows (may be none)
    const int xi = min(xw + j, rows - 1), in = xi / a.G, head = xi - in * a.G, tok = s0 + in;
    const bool valid = j < mine;

    // ---- what the rows see: tokens below hi that are not below lo, or below sinks
    int hi, lo, thi, tlo, trow, hi_min, lo_max, whi, wlo, sinks = 0;
    if (a.mode == kRowsPrompt) {
        const int len = wave_uniform(rows_len(a, seg)), before = len - n;
        auto low = [&](int x) { return a.window > 0 ? max(x - a.window, 0) : 0; };
        sinks = a.window > 0 ? a.sinks : 0;
        hi = before + in + 1;
        lo = low(hi);
        thi = before + (min(x0 + Z::ROWS, rows) - 1) / a.G + 1;
        tlo = low(before + x0 / a.G + 1);
        hi_min = before + min(xw, rows - 1) / a.G + 1;
        whi = before + (min(xw + 32, rows) - 1) / a.G + 1;
        wlo = low(hi_min);
        lo_max = low(whi);
        trow = seg;
    } else if (a.mode == kRowsPrefix) {
        const int pre = wave_uniform(group_prefix(a, seg, s0));
        hi = min(rows_len(a, tok), pre);
        lo = tlo = wlo = lo_max = 0;
        thi = whi = pre;
        hi_min = __any(valid && hi < pre) ? 0 : pre;
        trow = s0;
    } else {
        const int g = wave_search(a.groups, seg, [&](int i) { return rows_start(a, i); });
        int pre = 0;
        if (g >= 0) {
            const int first = wave_uniform(rows_start(a, g)), end = wave_uniform(rows_start(a, g + 1));
            if (seg < end) pre = wave_uniform(group_prefix(a, g, first));
        }
        hi = thi = whi = hi_min = wave_uniform(rows_len(a, seg));
        lo = tlo = wlo = lo_max = min(pre, thi);
        trow = seg;
    }
    if (!valid) {  // (rows that nobody asks for never make a block an edge)
        hi = INT_MAX;
        lo = 0;
    }

    // ---- the tile's blocks: those of the first tokens that stay visible, then
    // from tlo on; this piece takes its share of them
    const int base0 = tlo & ~7;
    int first_blocks = sinks > 0 ? (min(sinks, tlo) + BT - 1) / BT : 0;
    const bool apart = first_blocks * BT < base0;
    if (!apart) first_blocks = 0;
    const int base = apart || sinks == 0 ? base0 : 0;
    const int blocks = thi > base ? first_blocks + (thi - base + BT - 1) / BT : 0;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * piece / a.pieces);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (piece + 1) / a.pieces);
    const int last_group = max(thi - 1, 0) & ~7;
    auto block_at = [&](int b) { return b < first_blocks ? b * BT : base + (b - first_blocks) * BT; };

    // ---- copies: lane's place in a group's keys, pieces exchanged
    uint32_t koff[Z::IPG];
#pragma unroll
    for (int i = 0; i < Z::IPG; ++i) {
        const int p = i * 64 + lane, r = p / CN, c = p - r * CN;
        koff[i] = r * (Dp * ES) + ((c ^ Z::swizzle(8 * (RW == 4 ? wave : 0) + r)) << 4);
    }
    const int32_t* trow_at = a.table + static_cast<size_t>(trow) * a.table_stride;
    uint8_t* const team = s_mem + (RW == 4 ? 0 : wave * 2 * Z::STAGE);
    auto copy = [&](int b, int stage) __attribute__((always_inline)) {
        uint8_t* dst = team + stage * Z::STAGE;
        const int s = block_at(b);
#pragma unroll
        for (int u = 0; u < Z::GROUPS; ++u) {
            const int g = RW == 4 ? wave + W * u : u;
            const int t = min(s + 8 * g, last_group);
            const int pg = scalar_i32(trow_at, static_cast<uint32_t>(t) >> a.page_shift);
            const uint32_t p = static_cast<uint32_t>(pg) < static_cast<uint32_t>(a.pages) ? pg : 0;
            const size_t row = ((static_cast<size_t>(p) * a.H + hk) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
            const uint8_t* at = a.cache + row * (Dp * ES);
            const auto rk = buffer_rsrc(at, Z::GB), rv = buffer_rsrc(at + a.off_v, Z::GB);
#pragma unroll
            for (int i = 0; i < Z::IPG; ++i) {
                if (Z::GB % 1024 == 0 || i + 1 < Z::IPG || lane < (Z::GB % 1024) / 16) {
                    const uint32_t ko = RW == 4 || u % 2 == 0 ? koff[i] : koff[i] ^ Z::ODD;
                    buffer_copy_lds16(rk, dst + g * Z::GB + i * 1024, ko);
                    buffer_copy_lds16(rv, dst + Z::KB + g * Z::GB + i * 1024, (i * 64 + lane) * 16);
                }
            }
            if constexpr (I8) {
                const auto rks = buffer_rsrc(a.cache + a.off_ks + row * 4, 32), rvs = buffer_rsrc(a.cache + a.off_vs + row * 4, 32);
                if (lane < 8) {
                    copy_lds4(rks, dst + 2 * Z::KB + g * 64, lane * 4);
                    copy_lds4(rvs, dst + 2 * Z::KB + g * 64 + 32, lane * 4);
                }
            }
        }
    };
    const int bstep = RW == 4 ? 1 : W, bfirst = b0 + (RW == 4 ? 0 : wave);
    if (bfirst < b1) copy(bfirst, 0);

    // ---- the rows' queries: operand kc holds 8 elements of the lane's row
    bf16x8_t qf[NQ][2 * NC];
    const int64_t qat = static_cast<int64_t>(tok) * a.q_stride + (static_cast<int64_t>(hk) * a.G + head) * a.D;
    auto queries = [&](auto load) __attribute__((always_inline)) {
#pragma unroll
        for (int kc = 0; kc < 2 * NC; ++kc) {
            const int d = I8 ? 32 * (kc / 2) + 16 * h + 8 * (kc % 2) : 16 * kc + 8 * h;
            float f[8];
            load(d, valid && d < a.D, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = a.negative ? -f[e] : f[e];
            bf16x8_t t[NQ];
            rows_terms<NQ>(f, t);
#pragma unroll
            for (int q = 0; q < NQ; ++q) qf[q][kc] = t[q];
        }
    };
    // (places without an element read the row's first ones, and use none of them)
    const uint8_t* qp = static_cast<const uint8_t*>(a.q) + qat * (a.q32 ? 4 : 2);
    if (a.qvec && F32 && a.q32) {
        queries([&](int d, bool some, float (&f)[8]) __attribute__((always_inline)) {
            const uint4* p = reinterpret_cast<const uint4*>(qp + (some ? 4 * d : 0));
            const uint4 u = p[0], v = p[1];
            const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = some ? __uint_as_float(w[e]) : 0.0f;
        });
    } else if (a.qvec) {
        queries([&](int d, bool some, float (&f)[8]) __attribute__((always_inline)) {
            const uint4 u = *reinterpret_cast<const uint4*>(qp + (some ? 2 * d : 0));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = some ? __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16) : 0.0f;
        });
    } else {
        queries([&](int d, bool some, float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = load_act(qp, a.q32 ? BITQ_DT_F32 : BITQ_DT_BF16, min(d + e, a.D - 1));
                f[e] = some && d + e < a.D ? v : 0.0f;
            }
        });
    }

    f32x16_t o[NC];
#pragma unroll
    for (int d = 0; d < NC; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float m = -FLT_MAX, l = 0.0f;  // m in powers of two: p = 2^(c x - m)

    const int kr = 16 * (j >> 4) + 8 * ((j >> 2) & 1) + 4 * ((j >> 3) & 1) + (j & 3);  // token of row j of a score tile
    const int krow = kr * (Dp * ES), ksw = Z::swizzle(kr);

    auto compute = [&](int s, int stage, bool edge) __attribute__((always_inline)) {
        const uint8_t* st = team + stage * Z::STAGE;
        float x[8 * T16];
        // ---- scores of tokens s + 16 t + 8 h + e
#pragma unroll
        for (int kt = 0; kt < BT / 32; ++kt) {
            f32x16_t acc;
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
            if constexpr (!I8) {
#pragma unroll
                for (int kc = 0; kc < 2 * NC; ++kc) {
                    const bf16x8_t kf = *reinterpret_cast<const bf16x8_t*>(st + kt * 32 * Dp * ES + krow + (((2 * kc + h) ^ ksw) << 4));
#pragma unroll
                    for (int q = NQ - 1; q >= 0; --q) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[q][kc], acc, 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int kp = 0; kp < NC; ++kp) {
                    const uint4 u = *reinterpret_cast<const uint4*>(st + kt * 32 * Dp * ES + krow + (((2 * kp + h) ^ ksw) << 4));
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const bf16x8_t kf = b ? rows_codes(u.z, u.w) : rows_codes(u.x, u.y);
#pragma unroll
                        for (int q = NQ - 1; q >= 0; --q)
                            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[q][2 * kp + b], acc, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * kt + e] = acc[e];
        }
        const float* sc = reinterpret_cast<const float*>(st + 2 * Z::KB);
        if constexpr (I8) {
#pragma unroll
            for (int t = 0; t < T16; ++t) {
                const f32x4_t k0 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16);
                const f32x4_t k1 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16 + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[8 * t + e] *= k0[e];
                    x[8 * t + 4 + e] *= k1[e];
                }
            }
        }
        uint32_t keep = ~0u;  // bit 8 t + e: the row sees that token
        if (edge) {
            keep = 0;
#pragma unroll
            for (int i = 0; i < 8 * T16; ++i) {
                const int tk = s + 16 * (i / 8) + 8 * h + i % 8;
                const bool see = tk < hi && (tk >= lo || tk < sinks);
                keep |= see ? 1u << i : 0u;
                x[i] = see ? x[i] : -INFINITY;
            }
        }
        // ---- weights
        float mx = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < 8 * T16; ++i) mx = fmaxf(mx, x[i]);
        mx = fmaxf(pair_max(mx) * a.c, -FLT_MAX);
        if (__any(mx > m + 8.0f)) {  // (each row by its own maximum: its result depends on no other row)
            const float mn = mx > m + 8.0f ? mx : m, f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < NC; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= f;
        }
#pragma unroll
        for (int i = 0; i < 8 * T16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], a.c, -m));
            l += x[i];
        }
        if constexpr (I8) {
#pragma unroll
            for (int t = 0; t < T16; ++t) {
                const f32x4_t v0 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16 + 8);
                const f32x4_t v1 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16 + 12);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = x[8 * t + e] * (e < 4 ? v0[e & 3] : v1[e & 3]);
                    x[8 * t + e] = !edge || (keep >> (8 * t + e) & 1) ? w : 0.0f;  // (scales of hidden tokens may be anything)
                }
            }
        }
        // ---- values
        bool odd = false;  // edges, bf16: some value of the block is not finite
#pragma unroll
        for (int t = 0; t < T16; ++t) {
            bf16x8_t pf[NP];
            rows_terms<NP>(x + 8 * t, pf);
#pragma unroll
            for (int d = 0; d < NC; ++d) {
                bf16x8_t vf;
                const uint8_t* vp = st + Z::KB + ((2 * t + h) * Dp + 32 * d + j) * (8 * ES);
                if constexpr (I8) {
                    const uint2 u = *reinterpret_cast<const uint2*>(vp);
                    vf = rows_codes(u.x, u.y);
                } else {
                    uint4 u = *reinterpret_cast<const uint4*>(vp);
                    if (edge) {  // a hidden value times a weight of 0 must be 0: what is not finite counts as 0 here, and below
                        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool a0 = (w[e] & 0x7F80u) == 0x7F80u, a1 = (w[e] & 0x7F800000u) == 0x7F800000u;
                            odd = odd || a0 || a1;
                            w[e] &= (a0 ? 0xFFFF0000u : ~0u) & (a1 ? 0x0000FFFFu : ~0u);
                        }
                        u = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    vf = __builtin_bit_cast(bf16x8_t, u);
                }
#pragma unroll
                for (int q = NP - 1; q >= 0; --q) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[q], o[d], 0, 0, 0);
            }
        }
        if constexpr (!I8) {
            if (edge && __any(odd)) {
                // rows that see a value that is not finite get NaN in its element: count them with the same product
#pragma unroll
                for (int d = 0; d < NC; ++d) {
                    f32x16_t cnt;
#pragma unroll
                    for (int e = 0; e < 16; ++e) cnt[e] = 0.0f;
#pragma unroll
                    for (int t = 0; t < T16; ++t) {
                        const uint4 u = *reinterpret_cast<const uint4*>(st + Z::KB + ((2 * t + h) * Dp + 32 * d + j) * (8 * ES));
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                        bf16x8_t vf, pf;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t b = e & 1 ? w[e >> 1] >> 16 : w[e >> 1];
                            vf[e] = static_cast<__bf16>((b & 0x7F80u) == 0x7F80u ? 1.0f : 0.0f);
                            pf[e] = static_cast<__bf16>(keep >> (8 * t + e) & 1 ? 1.0f : 0.0f);
                        }
                        cnt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, cnt, 0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[d][e] = cnt[e] > 0.0f ? __builtin_nanf("") : o[d][e];
                }
            }
        }
    };

    int stage = 0;
    for (int b = bfirst; b < b1; b += bstep) {
        const int s = block_at(b);
        rows_wait_copies<0>();
        if constexpr (RW == 4) {
            rows_wait_lds();
            __builtin_amdgcn_s_barrier();  // every wave's copies have landed, and the other stage is read no more
            asm volatile("" ::: "memory");
        } else {
            rows_wait_lds();
        }
        if (b + bstep < b1) copy(b + bstep, stage ^ 1);
        const bool any = mine > 0 && s < whi && (s + BT > wlo || s < sinks);
        if (any) {
            const bool all = s + BT <= hi_min && (s >= lo_max || s + BT <= sinks);
            if (all) compute(s, stage, false);
            else compute(s, stage, true);
        }
        stage ^= 1;
    }

    // ---- results
    l = pair_sum(l);
    const size_t row_at = static_cast<size_t>(tok) * a.A + static_cast<size_t>(hk) * a.G + head;
    if constexpr (RW == 4) {
        if (!valid) return;
        if (a.all == 0) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int d = 0; d < NC; ++d)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    rows_store4(a, row_at * a.D, 32 * d + 8 * b + 4 * h,
                                f32x4_t{o[d][4 * b] * inv, o[d][4 * b + 1] * inv, o[d][4 * b + 2] * inv, o[d][4 * b + 3] * inv});
            if (h == 0 && a.lse) a.lse[row_at] = rows_lse(m, l);
        } else {
            const size_t at = row_at * a.all + a.piece0 + piece;
            if (b0 < b1) {
#pragma unroll
                for (int d = 0; d < NC; ++d)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        *reinterpret_cast<f32x4_t*>(a.part + at * Dp + 32 * d + 8 * b + 4 * h) =
                            f32x4_t{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
            }
            if (h == 0) a.ml[at] = make_float2(m, l);
        }
    } else {
        rows_wait_lds();
        __syncthreads();  // (every wave has read its blocks: the stages' place is free)
        float* so = reinterpret_cast<float*>(s_mem) + wave * 32 * (Z::ORow + 2);
        float *sm = so + 32 * Z::ORow, *sl = sm + 32;
#pragma unroll
        for (int d = 0; d < NC; ++d)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                *reinterpret_cast<f32x4_t*>(so + j * Z::ORow + 32 * d + 8 * b + 4 * h) =
                    f32x4_t{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
        if (h == 0) {
            sm[j] = m;
            sl[j] = l;
        }
        __syncthreads();
        const float* all_o = reinterpret_cast<const float*>(s_mem);
        constexpr int WS = 32 * (Z::ORow + 2);
        for (int i = tid; i < mine * (Dp / 4); i += 64 * W) {
            const int r = i / (Dp / 4), d = 4 * (i - r * (Dp / 4));
            float M = -FLT_MAX, L = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) M = fmaxf(M, all_o[v * WS + 32 * Z::ORow + r]);
            f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const float f = __builtin_amdgcn_exp2f(all_o[v * WS + 32 * Z::ORow + r] - M);
                L += f * all_o[v * WS + 32 * Z::ORow + 32 + r];
                const f32x4_t u = *reinterpret_cast<const f32x4_t*>(all_o + v * WS + r * Z::ORow + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += f * u[e];
            }
            const int x = xw + r, ti = x / a.G;
            const size_t ra = static_cast<size_t>(s0 + ti) * a.A + static_cast<size_t>(hk) * a.G + (x - ti * a.G);
            if (a.all == 0) {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                rows_store4(a, ra * a.D, d, f32x4_t{acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv});
                if (d == 0 && a.lse) a.lse[ra] = rows_lse(M, L);
            } else {
                const size_t at = ra * a.all + a.piece0 + piece;
                if (b0 < b1) *reinterpret_cast<f32x4_t*>(a.part + at * Dp + d) = acc;
                if (d == 0) a.ml[at] = make_float2(M, L);
            }
        }
    }
}

}  // namespace bitq
