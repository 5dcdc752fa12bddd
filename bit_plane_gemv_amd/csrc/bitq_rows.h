// Attention of several query rows over the paged cache of libbitq: the kernel
// of bitq_prompt_attn and bitq_shared_attn, compiled per cache type in
// bitq_rows_bf16.hip and bitq_rows_int8.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

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
// stages of them, one in flight while the other is worked on.  Copies are issued
// between the products (in a row before them: the same 250 us for a prompt of 4096
// tokens, 113 against 111 us for 64 requests on a prefix of 16384).  They move
// groups of 8 tokens (a page has whole groups), so a page's index is the same
// for a whole copy instruction.  Keys are stored with their 16-byte pieces
// exchanged within a row by the row's number, so that the reads of a score tile
// (one piece of 32 rows) fall on all banks alike.
//   RW = 4: 128 rows, 32 to each of the 4 waves, which share blocks of 64 tokens
//           (an int8 block is turned into bf16 once for all of them).
//   RW = 1: 32 rows; each wave takes every W-th block of 32 tokens for itself
//           (no meeting of the waves until the end), and the waves' results are
//           joined in LDS.  For few rows, where the memory is the bound.
// A tile's tokens may be split over `pieces` workgroups; rows_join_kernel joins.
//
// Bound: RW = 1 by the memory (64 single tokens in a window of 2048, 64 heads on 8
// of 128, bf16: 100 us, 5.4 TB/s).  RW = 4 by the products and the softmax beside
// them: a prompt of 4096 tokens, 32 heads of 128 on 8, bf16, 239 to 250 us by the
// card's clock, 576 TFLOP/s of the formula's products, 1150 with the three terms
// of p (a large library product: 1426).  Of a block of 64 tokens x 32 rows the
// products take 2048 cycles of a SIMD, its 357 vector instructions some 1430; two
// waves share it, and a product is under way in 54 % of the cycles.  With two
// terms of p, and taken out for comparison, us of 217 at that time: the copies 23,
// exponentials 13, three quarters of the softmax 24, LDS reads 6; one wave a SIMD:
// 340 us.
//
// Precision.  Cache rows are exact in bf16; int8 scales are applied in fp32, to
// the scores and to p.  fp32 q is split into 3 bf16 terms, which hold its 24
// bits, and so is p (times V's scale), whatever the type of the outputs: with 2
// terms, which err by up to 2^-17 of each weight, an output that is a small
// difference of large terms loses bits that its own rounding would have kept,
// and one bf16 output in a thousand rounds to its other neighbour.
// m follows the maximum only when it has grown by more than 2^8 (p may then be
// up to 2^8), which changes no result while sums stay in fp32's range.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

enum RowsMode { kRowsPrompt = 0, kRowsPrefix = 1, kRowsOwn = 2 };  // of a workgroup

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
    int R, T;              // requests, rows of q (shared: one a request)
    int H, A, G, D, page_shift, pages, table_stride, max_len, window, sinks, max_prefix;
    int groups;            // of requests with a common prefix (0: bitq_prompt_attn)
    int tiles, pieces;     // places for tiles (an upper bound of the tiles) and pieces that each is split into
    int own_tiles, own_pieces, tps;  // shared: those of the requests' own tokens, and its tiles per request
    int all;               // partial results of a row, a prefix's pieces first; 0: no split
    float c;               // |scale| log2(e) (> 0); a negative scale turns q's sign
    bool negative, qvec, ovec;
    int odt;
};

template <int KVT, int NC, bool Q32, int RW>
struct RowsShape {
    static constexpr bool I8 = KVT == BITQ_KV_INT8;
    static constexpr int Dp = 32 * NC, ES = I8 ? 1 : 2;
    static constexpr int W = rows_waves(RW);
    static constexpr int BT = rows_block(RW);  // tokens of a block
    static constexpr int ROWS = 32 * RW;
    static constexpr int NQ = Q32 ? 3 : 1, NP = 3;
    static constexpr int KB = BT * Dp * ES, STAGE = 2 * KB + (I8 ? 8 * BT : 0);
    static constexpr int TEAMS = RW == 4 ? 1 : W;
    static constexpr int GROUPS = BT / 8 / (RW == 4 ? W : 1);  // groups of 8 tokens that a wave copies
    static constexpr int GB = 8 * Dp * ES, IPG = (GB + 1023) / 1024;
    static constexpr int COPIES = GROUPS * (2 * IPG + (I8 ? 2 : 0));
    static constexpr int CN = Dp * ES / 16;                   // 16-byte pieces of a key
    static constexpr int ORow = Dp + 4;                       // floats of a row when the waves' results meet
    static constexpr int JOIN = RW == 4 ? 0 : W * 32 * (ORow + 2) * 4;
    static constexpr int LDS = rows_lds(KVT, NC, RW);
    // int8 rows of RW = 4 are turned into bf16 once for all waves, in LDS behind the stages; with RW = 1 each wave turns its
    // own operands
    static constexpr bool CONV = I8 && RW == 4, C8 = I8 && !CONV;
    static constexpr int OES = C8 ? 1 : 2, OKB = BT * Dp * OES, OCN = Dp * OES / 16;  // as read by the products
    static_assert(LDS >= TEAMS * 2 * STAGE + (CONV ? 2 * OKB : 0) && LDS >= JOIN, "stages, then the waves' results");
    // Piece c of row r is stored at piece c ^ swizzle(r), so that any 16 rows that differ in their last 4 bits have a
    // piece in 16 different sixteenths of the banks (256 bytes); rows 8 further on differ in ODD of a piece's offset.
    static constexpr __device__ __forceinline__ int swizzle_of(int cn, int r) {
        return cn % 16 == 0 ? r & 15 : cn % 8 == 0 ? (r >> 1) & 7 : cn % 4 == 0 ? (r >> 2) & 3 : (r >> 3) & 1;
    }
    static constexpr __device__ __forceinline__ int swizzle(int r) { return swizzle_of(CN, r); }
    static constexpr uint32_t ODD = CN % 16 == 0 ? 128 : CN % 8 == 0 ? 64 : CN % 4 == 0 ? 32 : 16;
};

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
// 16 (4) bytes per lane from memory straight into LDS, lane l's at dst + 16 l
// (4 l).  Written as instructions: the compiler, which cannot tell the stage that
// is copied into from the one that is read, would wait for the copy before every
// LDS read behind the builtin.  The kernel waits for its copies itself
// (rows_wait_copies), and instructions that the compiler does not count only make
// the waits that it adds for its own loads longer.  No registers are written.
// (s_nop: a scalar written by a vector instruction is ready for a buffer
// instruction after 5 cycles, and M0 after 1)
__device__ __forceinline__ u32x4_t rows_rsrc(uint64_t a, uint32_t bytes) {
    u32x4_t r;
    r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32)) & 0xFFFFu;
    r[2] = bytes;
    r[3] = 0x00020000u;  // (as in buffer_rsrc)
    return r;
}
__device__ __forceinline__ uint32_t rows_lds_address(const uint8_t* shared) {
#if defined(__HIP_DEVICE_COMPILE__)
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)shared));
#else
    return 0;
#endif
}
template <int BYTES>
__device__ __forceinline__ void rows_copy_lds(u32x4_t rsrc, uint32_t dst, uint32_t voff) {
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(voff), "s"(rsrc) : "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(at), "v"(voff), "s"(rsrc) : "m0");
#endif
}

// two elements as bf16, by one instruction
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t rows_round2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// 8 int8 codes as bf16 (exact)
__device__ __forceinline__ bf16x8_t rows_codes(uint32_t lo, uint32_t hi) {
    const uint32_t b[2] = {lo, hi};
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = b[e >> 1] >> (16 * (e & 1));
        w[e] = rows_round2(static_cast<float>(static_cast<int>(static_cast<int8_t>(u))),
                           static_cast<float>(static_cast<int>(static_cast<int8_t>(u >> 8))));
    }
    return __builtin_bit_cast(bf16x8_t, make_uint4(w[0], w[1], w[2], w[3]));
}

// x = sum of the N bf16 terms, each the rounding of what the ones before leave
template <int N>
__device__ __forceinline__ void rows_terms(const float* x, bf16x8_t (&t)[N]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = rows_round2(r[2 * e], r[2 * e + 1]);
            if (n + 1 < N) {
                r[2 * e] -= __uint_as_float(w[e] << 16);
                r[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
        t[n] = __builtin_bit_cast(bf16x8_t, make_uint4(w[0], w[1], w[2], w[3]));
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
// elements d .. d + 3 of an output row (i: element 0 of the row)
__device__ __forceinline__ void rows_store4(const RowsArgs& a, size_t i, int d, f32x4_t v) {
    if (a.ovec) {  // (D a multiple of 8)
        if (d >= a.D) return;
        if (a.odt == BITQ_DT_F32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + i + d) = v;
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + i + d) = make_uint2(rows_round2(v[0], v[1]), rows_round2(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < a.D) rows_store(a, i + d + e, v[e]);
    }
}
__device__ __forceinline__ float rows_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

template <int KVT, int NC, bool Q32, int RW>
__global__ __launch_bounds__(64 * rows_waves(RW), (rows_groups_per_cu(KVT, NC, Q32, RW) * rows_waves(RW) + 3) / 4) void rows_attn_kernel(RowsArgs a) {
    using Z = RowsShape<KVT, NC, Q32, RW>;
    constexpr bool I8 = Z::I8, C8 = Z::C8;
    constexpr int Dp = Z::Dp, ES = Z::ES, W = Z::W, BT = Z::BT, NQ = Z::NQ, NP = Z::NP, CN = Z::CN, T16 = BT / 16;
    __shared__ __align__(16) uint8_t s_mem[Z::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6), h = lane >> 5, j = lane & 31;

    // ---- the tile: heads fastest (an XCD, blockIdx % 8, then sees few heads and
    // shares their keys in its L2), last tiles first (a prompt's longest)
    // (a launch with prefixes and the requests' own tokens: their workgroups alternate)
    uint32_t id = blockIdx.x;
    int mode = kRowsPrompt, tiles = a.tiles, pieces = a.pieces, piece0 = 0, segments = a.R;
    if (a.groups > 0) {
        const uint32_t n1 = static_cast<uint32_t>(a.tiles) * a.pieces * a.H;
        const uint32_t before = static_cast<uint32_t>(static_cast<uint64_t>(id) * n1 / gridDim.x);
        const uint32_t after = static_cast<uint32_t>(static_cast<uint64_t>(id + 1) * n1 / gridDim.x);
        if (after > before) {
            mode = kRowsPrefix;
            id = before;
            segments = a.groups;
        } else {
            mode = kRowsOwn;
            id -= before;
            tiles = a.own_tiles;
            piece0 = a.pieces;
            pieces = a.own_pieces;
        }
    }
    const uint32_t rest = id / static_cast<uint32_t>(a.H);
    const int hk = id - rest * a.H, slot = tiles - 1 - static_cast<int>(rest / static_cast<uint32_t>(pieces));
    const int piece = rest % static_cast<uint32_t>(pieces);
    int seg, tile, s0, n;  // segment, tile of it, its first row token and their number
    int len0 = 0;          // the segment's length (kRowsPrompt, kRowsOwn) or its first request's
    int g0 = -1, gend = 0, gpre = 0;  // kRowsOwn: first and last request and prefix of the request's group (g0 < 0: none)
    if (mode == kRowsOwn) {
        seg = slot / a.tps;
        tile = slot - seg * a.tps;
        s0 = seg;
        n = 1;
        // (up to 63 segments or groups: their starts, lengths and prefixes are loaded together, a lane each)
        const int len_v = rows_len(a, seg);
        if (a.groups < 64) {
            const int v = rows_start(a, min(lane, a.groups)), pv = a.prefix[min(lane, a.groups - 1)];
            const int c = __builtin_popcountll(__ballot(lane < a.groups && v <= seg));
            if (c > 0) {
                g0 = __builtin_amdgcn_readlane(v, c - 1);
                gend = __builtin_amdgcn_readlane(v, c);
                gpre = __builtin_amdgcn_readlane(pv, c - 1);
            }
        } else {
            const int g = wave_search(a.groups, seg, [&](int i) { return rows_start(a, i); });
            if (g >= 0) {
                g0 = wave_uniform(rows_start(a, g));
                gend = wave_uniform(rows_start(a, g + 1));
                gpre = wave_uniform(a.prefix[g]);
            }
        }
        len0 = wave_uniform(len_v);
        if (g0 > seg || seg >= gend) g0 = -1;  // (later groups: only where starts do not ascend)
    } else {
        // the tiles of segment r lie from floor(start[r] G / ROWS) + r on: ceil(n G / ROWS) of them always fit
        auto place = [&](int start, int r) { return start * a.G / Z::ROWS + r; };
        int s1;
        if (segments < 64) {
            const int v = rows_start(a, min(lane, segments));
            const int len_v = mode == kRowsPrompt ? rows_len(a, min(lane, segments - 1)) : 0;
            const int c = __builtin_popcountll(__ballot(lane < segments && place(v, lane) <= slot));
            if (c == 0) return;
            seg = c - 1;
            s0 = __builtin_amdgcn_readlane(v, seg);
            s1 = __builtin_amdgcn_readlane(v, c);
            len0 = __builtin_amdgcn_readlane(len_v, seg);
        } else {
            seg = wave_search(segments, slot, [&](int r) { return place(rows_start(a, r), r); });
            if (seg < 0) return;
            seg = wave_uniform(seg);
            s0 = wave_uniform(rows_start(a, seg));
            s1 = wave_uniform(rows_start(a, seg + 1));
            if (mode == kRowsPrompt) len0 = wave_uniform(rows_len(a, seg));
        }
        n = s1 - s0;
        tile = slot - place(s0, seg);
        if (n <= 0 || tile < 0 || tile * Z::ROWS >= n * a.G) return;
    }
    const int rows = n * a.G, x0 = tile * Z::ROWS;
    const int xw = x0 + (RW == 4 ? 32 * wave : 0), mine = min(32, rows - xw);  // this wave's rows (may be none)
    const int xi = min(xw + j, rows - 1), in = xi / a.G, head = xi - in * a.G, tok = s0 + in;
    const bool valid = j < mine;

    // ---- what the rows see: tokens below hi that are not below lo, or below sinks
    int hi, lo, thi, tlo, trow, hi_min, lo_max, whi, wlo, sinks = 0;
    if (mode == kRowsPrompt) {
        const int before = len0 - n;
        auto low = [&](int x) { return a.window > 0 && x > a.window ? x - a.window : 0; };  // (x may be negative)
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
    } else if (mode == kRowsPrefix) {
        const int pre = wave_uniform(group_prefix(a, seg, s0));
        hi = min(rows_len(a, tok), pre);
        lo = tlo = wlo = lo_max = 0;
        thi = whi = pre;
        hi_min = __any(valid && hi < pre) ? 0 : pre;
        trow = s0;
    } else {
        const int pre = g0 >= 0 ? min(min(max(gpre, 0), a.max_prefix), wave_uniform(rows_len(a, g0))) : 0;
        hi = thi = whi = hi_min = len0;
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
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * piece / pieces);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (piece + 1) / pieces);
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
    // Pages of a block's groups, a lane each, loaded a block ahead: its copies then wait for no table.  (Any block: tokens past
    // the last group are its own.)
    int pages = 0;
    auto look_up = [&](int b) __attribute__((always_inline)) {
        pages = trow_at[static_cast<uint32_t>(min(block_at(b) + 8 * (lane & (BT / 8 - 1)), last_group)) >> a.page_shift];
    };
    // A block's copies: the groups' places, then one instruction at a time, so that they can be issued between products (a
    // row of them holds the wave up for 150 cycles each).
    const uint8_t* const kbase = a.cache + ((static_cast<size_t>(hk) << a.page_shift) * (Dp * ES));  // this head's keys in page 0
    const uint32_t page_bytes = (static_cast<uint32_t>(a.H) << a.page_shift) * (Dp * ES);             // (<= 2^29)
    const uint32_t team_lds = rows_lds_address(s_mem) + (RW == 4 ? 0 : wave * 2 * Z::STAGE);
    const int page_mask = (1 << a.page_shift) - 1, pool = a.pages;
    const size_t off_v = a.off_v;
    uint64_t ck[Z::GROUPS];  // places of the groups' keys (values: off_v further on)
    uint32_t cdst = 0;
    auto aim = [&](int b, int stage) __attribute__((always_inline)) {
        cdst = team_lds + stage * Z::STAGE;
        // (a lane for each group, then into scalar registers)
        const int t = min(block_at(b) + 8 * (lane & (BT / 8 - 1)), last_group);
        const uint32_t p = static_cast<uint32_t>(pages) < static_cast<uint32_t>(pool) ? pages : 0;
        const uint64_t at = reinterpret_cast<uint64_t>(kbase) + static_cast<uint64_t>(p) * page_bytes +
                            static_cast<uint32_t>(t & page_mask) * (Dp * ES);
#pragma unroll
        for (int u = 0; u < Z::GROUPS; ++u) {
            const int g = RW == 4 ? wave + W * u : u;
            ck[u] = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(at), g)) |
                    static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(at >> 32), g))) << 32;
        }
    };
    auto copy_one = [&](int n) __attribute__((always_inline)) {  // n-th of COPIES
        constexpr int PER = Z::COPIES / Z::GROUPS;
        const int u = n / PER, i = n % PER, g = RW == 4 ? wave + W * u : u;
        const bool v = i & 1;
        if (i < 2 * Z::IPG) {
            const int part = i >> 1;
            // (the odd groups' keys differ in the swizzle's bit 3 of the row)
            const uint32_t off = v ? (part * 64 + lane) * 16 : RW == 4 || u % 2 == 0 ? koff[part] : koff[part] ^ Z::ODD;
            if (Z::GB % 1024 == 0 || part + 1 < Z::IPG || lane < (Z::GB % 1024) / 16)
                rows_copy_lds<16>(rows_rsrc(ck[u] + (v ? off_v : 0), Z::GB), cdst + (v ? Z::KB : 0) + g * Z::GB + part * 1024, off);
        } else if (lane < 8) {  // (a scale of 4 bytes for a row of Dp codes)
            const uint64_t row = (ck[u] - reinterpret_cast<uint64_t>(a.cache)) / Dp * 4;
            rows_copy_lds<4>(rows_rsrc(reinterpret_cast<uint64_t>(a.cache) + (v ? a.off_vs : a.off_ks) + row, 32),
                             cdst + 2 * Z::KB + g * 64 + (v ? 32 : 0), lane * 4);
        }
    };
    auto copy_all = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < Z::COPIES; ++i) copy_one(i);
    };
    const int bstep = RW == 4 ? 1 : W, bfirst = b0 + (RW == 4 ? 0 : wave);
    if (bfirst < b1) {
        look_up(bfirst);
        aim(bfirst, 0);
        copy_all();
        look_up(bfirst + bstep);
    }

    // ---- the rows' queries: operand kc holds 8 elements of the lane's row
    bf16x8_t qf[NQ][2 * NC];
    const int64_t qat = static_cast<int64_t>(tok) * a.q_stride + (static_cast<int64_t>(hk) * a.G + head) * a.D;
    auto queries = [&](auto load) __attribute__((always_inline)) {
#pragma unroll
        for (int kc = 0; kc < 2 * NC; ++kc) {
            const int d = C8 ? 32 * (kc / 2) + 16 * h + 8 * (kc % 2) : 16 * kc + 8 * h;
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
    const uint8_t* qp = static_cast<const uint8_t*>(a.q) + qat * (Q32 ? 4 : 2);
    if (Q32 && a.qvec) {
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
                const float v = load_act(qp, Q32 ? BITQ_DT_F32 : BITQ_DT_BF16, min(d + e, a.D - 1));
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
    const int krow = kr * (Dp * Z::OES), ksw = Z::swizzle_of(Z::OCN, kr);

    // Which tokens of the block at s this lane's row sees: bit 8 t + e is token s + 16 t + 8 h + e.
    auto seen = [&](int s) __attribute__((always_inline)) {
        auto below = [&](int limit) __attribute__((always_inline)) {
            uint32_t bits = 0;
#pragma unroll
            for (int t = 0; t < T16; ++t) bits |= ((1u << min(max(limit - (s + 16 * t + 8 * h), 0), 8)) - 1u) << (8 * t);
            return bits;
        };
        return below(hi) & (~below(lo) | below(sinks));
    };
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    typedef typename std::conditional<C8, u32x2_t, u32x4_t>::type Value;
    // One block.  The products and the softmax's instructions run side by side:
    // a wave's weights of 16 tokens are made while the matrix cores multiply the 16
    // before them, and operands are read from LDS well before they are needed.
    auto compute = [&](int s, int stage, bool edge, auto copies) __attribute__((always_inline)) {
        const uint8_t* st = team + stage * Z::STAGE;
        const float* sc = reinterpret_cast<const float*>(st + 2 * Z::KB);
        const uint8_t* ob = Z::CONV ? s_mem + 2 * Z::STAGE : st;  // operands
        auto value = [&](int t, int d) __attribute__((always_inline)) {  // operand: elements 32 d + j of tokens 16 t + 8 h ..
            return *reinterpret_cast<const Value*>(ob + Z::OKB + ((2 * t + h) * Dp + 32 * d + j) * (8 * Z::OES));
        };
        auto operand = [&](Value u) __attribute__((always_inline)) {
            if constexpr (C8) return rows_codes(u[0], u[1]);
            else return __builtin_bit_cast(bf16x8_t, u);
        };
        // ---- scores of tokens s + 16 t + 8 h + e
        constexpr int KT = BT / 32, KR = C8 ? NC : 2 * NC;  // score tiles, and reads of a tile's keys
        constexpr int KN = KR * KT, AHEAD = KN < 8 ? KN : 8;
        f32x16_t acc[KT];
        u32x4_t kf[KN];
        auto key = [&](int i) __attribute__((always_inline)) {
            kf[i] = *reinterpret_cast<const u32x4_t*>(ob + (i % KT) * 32 * Dp * Z::OES + krow + (((2 * (i / KT) + h) ^ ksw) << 4));
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) key(i);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int kt = i % KT, kr_ = i / KT;
#pragma unroll
            for (int b = 0; b < (C8 ? 2 : 1); ++b) {
                const bf16x8_t k8 = !C8 ? __builtin_bit_cast(bf16x8_t, kf[i])
                                    : b ? rows_codes(kf[i][2], kf[i][3]) : rows_codes(kf[i][0], kf[i][1]);
#pragma unroll
                for (int q = NQ - 1; q >= 0; --q) {
                    const f32x16_t zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                    acc[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, qf[q][C8 ? 2 * kr_ + b : kr_],
                                                                      kr_ == 0 && b == 0 && q == NQ - 1 ? zero : acc[kt], 0, 0, 0);
                }
            }
            if (i + AHEAD < KN) key(i + AHEAD);
            if constexpr (decltype(copies)::value) {
#pragma unroll
                for (int n = Z::COPIES * i / KN; n < Z::COPIES * (i + 1) / KN; ++n) copy_one(n);
            }
        }
        Value vf[2][NC];
#pragma unroll
        for (int d = 0; d < NC; ++d) vf[0][d] = value(0, d);
        float x[8 * T16];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * kt + e] = acc[kt][e];
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
        uint32_t keep = ~0u;
        if (edge) {
            asm volatile("");  // (a branch, not selects in every block)
            keep = seen(s);
#pragma unroll
            for (int i = 0; i < 8 * T16; ++i) {
                const uint32_t yes = static_cast<uint32_t>(static_cast<int32_t>(keep << (31 - i)) >> 31);
                x[i] = __uint_as_float((__float_as_uint(x[i]) & yes) | (0xFF800000u & ~yes));  // else -inf
            }
        }
        // ---- the running maximum.  (The wave that has products to issue goes first: 208 -> 199 us for a prompt of 4096, with two
        // terms of p.)
        __builtin_amdgcn_s_setprio(0);
        float mx = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < 8 * T16; ++i) mx = fmaxf(mx, x[i]);
        mx = fmaxf(pair_max(mx) * a.c, -FLT_MAX);
        // An exponent c x - m is rounded once, but m is the rounded maximum: the largest exponent is the rounding error of m, a
        // factor that all of a row's weights have in common while it is below 1.  Where scores are larger than 2^24 it could
        // take them out of range: such rows have x scaled and rounded before m is subtracted.
        const bool far = fabsf(mx) > 0x1p24f && mx > -FLT_MAX;
        float c = a.c;
        if (__any(far)) {
            asm volatile("");  // (a branch, not products in every block)
            const float f = far ? a.c : 1.0f;
            c = far ? 1.0f : a.c;
#pragma unroll
            for (int i = 0; i < 8 * T16; ++i) x[i] *= f;
        }
        if (__any(mx > m + 8.0f)) {  // (each row by its own maximum: its result depends on no other row)
            const float mn = mx > m + 8.0f ? mx : m, f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < NC; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= f;
        }
        // ---- weights of the t-th 16 tokens, as terms
        auto weights = [&](int t, bf16x8_t (&pf)[NP]) __attribute__((always_inline)) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[8 * t + e], c, -m));
            l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            if constexpr (I8) {
                const f32x4_t v0 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16 + 8);
                const f32x4_t v1 = *reinterpret_cast<const f32x4_t*>(sc + (2 * t + h) * 16 + 12);
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] *= e < 4 ? v0[e & 3] : v1[e & 3];
                if (edge) {  // (scales of hidden tokens may be anything)
                    asm volatile("");
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = __uint_as_float(__float_as_uint(p[e]) & static_cast<uint32_t>(static_cast<int32_t>(keep << (31 - 8 * t - e)) >> 31));
                }
            }
            rows_terms<NP>(p, pf);
        };
        bf16x8_t pf[2][NP];
        weights(0, pf[0]);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < T16; ++t) {
            if (t + 1 < T16) {
#pragma unroll
                for (int d = 0; d < NC; ++d) vf[(t + 1) & 1][d] = value(t + 1, d);
            }
            if (t + 1 < T16) weights(t + 1, pf[(t + 1) & 1]);
            bf16x8_t v[NC];
#pragma unroll
            for (int d = 0; d < NC; ++d) v[d] = operand(vf[t & 1][d]);
#pragma unroll
            for (int q = NP - 1; q >= 0; --q)  // (terms outside: a product does not wait for the one before it)
#pragma unroll
                for (int d = 0; d < NC; ++d) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[d], pf[t & 1][q], o[d], 0, 0, 0);
        }
    };

    // A hidden value times a weight of 0 must be 0: where a row does not see a token of a block, bf16 values that are not
    // finite (int8 codes always are) are looked for, and taken out of LDS, after the rows that see one have got NaN in its
    // element.
    // Whether some value of the part of the block that this wave looks after is not finite:
    constexpr int PART = Z::KB / 1024 / (RW == 4 ? W : 1);  // 16-byte pieces of a lane
    auto part_at = [&](int stage, int i) __attribute__((always_inline)) {
        return reinterpret_cast<u32x4_t*>(team + stage * Z::STAGE + Z::KB + (((RW == 4 ? wave : 0) * PART + i) * 64 + lane) * 16);
    };
    auto find_odd = [&](int stage) __attribute__((always_inline)) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < PART; ++i) {
            const u32x4_t w = *part_at(stage, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) most = max(most, max(w[e] & 0x7F80u, w[e] >> 16 & 0x7F80u));
        }
        return __any(most == 0x7F80u);
    };
    auto mark_odd = [&](int s, int stage) __attribute__((always_inline)) {  // (counted by a product)
        const uint32_t keep = seen(s);
#pragma unroll
        for (int d = 0; d < NC; ++d) {
            f32x16_t cnt = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
            for (int t = 0; t < T16; ++t) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(team + stage * Z::STAGE + Z::KB + ((2 * t + h) * Dp + 32 * d + j) * 16);
                bf16x8_t bad, see;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    bad[e] = static_cast<__bf16>((w[e >> 1] >> (16 * (e & 1)) & 0x7F80u) == 0x7F80u ? 1.0f : 0.0f);
                    see[e] = static_cast<__bf16>(keep >> (8 * t + e) & 1 ? 1.0f : 0.0f);
                }
                cnt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bad, see, cnt, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = cnt[e] > 0.0f ? __builtin_nanf("") : o[d][e];
        }
    };
    auto clear_odd = [&](int stage) __attribute__((always_inline)) {
#pragma unroll 1
        for (int i = 0; i < PART; ++i) {
            u32x4_t w = *part_at(stage, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = (w[e] & 0x7F80u) == 0x7F80u ? w[e] & 0xFFFF0000u : w[e];
                w[e] = (w[e] & 0x7F800000u) == 0x7F800000u ? w[e] & 0x0000FFFFu : w[e];
            }
            *part_at(stage, i) = w;
        }
    };
    // (edges of the tile: the waves of RW = 4 look for odd values together)
    const int tile_hi = mode != kRowsPrefix ? (mode == kRowsPrompt ? thi - (min(x0 + Z::ROWS, rows) - 1) / a.G + x0 / a.G : thi)
                        : RW == 4             ? (__syncthreads_or(hi_min < thi && mine > 0) ? 0 : thi)
                                              : hi_min;
    const int tile_lo = mode == kRowsPrompt && a.window > 0 ? (thi > a.window ? thi - a.window : 0) : lo_max;

    auto block = [&](int b, int stage, auto copies) __attribute__((always_inline)) {
        const int s = block_at(b);
        rows_wait_copies<0>();
        rows_wait_lds();
        if constexpr (RW == 4) {
            __builtin_amdgcn_s_barrier();  // every wave's copies have landed, and the other stage is read no more
            asm volatile("" ::: "memory");
        }
        if constexpr (decltype(copies)::value) {
            aim(b + bstep, stage ^ 1);
            look_up(b + 2 * bstep);
        }
        if constexpr (Z::CONV) {  // the codes as bf16, 16 of them at a time, with the keys' pieces exchanged anew
            const uint8_t* st = team + stage * Z::STAGE;
            uint8_t* ob = s_mem + 2 * Z::STAGE;
#pragma unroll
            for (int i = 0; i < (Z::KB / 16 + 64 * W - 1) / (64 * W); ++i) {
                const int at = i * 64 * W + tid;
                if (Z::KB / 16 % (64 * W) == 0 || at < Z::KB / 16) {
                    const u32x4_t k = *reinterpret_cast<const u32x4_t*>(st + at * 16);
                    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(st + Z::KB + at * 16);
                    const int r = at / CN, c = 2 * ((at - r * CN) ^ Z::swizzle(r)), sw = Z::swizzle_of(Z::OCN, r);
                    *reinterpret_cast<bf16x8_t*>(ob + r * (Dp * 2) + ((c ^ sw) << 4)) = rows_codes(k[0], k[1]);
                    *reinterpret_cast<bf16x8_t*>(ob + r * (Dp * 2) + (((c + 1) ^ sw) << 4)) = rows_codes(k[2], k[3]);
                    *reinterpret_cast<bf16x8_t*>(ob + Z::OKB + at * 32) = rows_codes(v[0], v[1]);
                    *reinterpret_cast<bf16x8_t*>(ob + Z::OKB + at * 32 + 16) = rows_codes(v[2], v[3]);
                }
            }
            rows_wait_lds();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        const bool any = mine > 0 && s < whi && (s + BT > wlo || s < sinks);
        if constexpr (!I8) {
            if (!(s + BT <= tile_hi && (s >= tile_lo || s + BT <= sinks))) {
                asm volatile("");
                bool odd = find_odd(stage);
                if constexpr (RW == 4) odd = __syncthreads_or(odd);
                if (odd) {
                    if (any) mark_odd(s, stage);
                    rows_wait_lds();
                    if constexpr (RW == 4) __syncthreads();
                    clear_odd(stage);
                    rows_wait_lds();
                    if constexpr (RW == 4) __syncthreads();
                }
            }
        }
        if (any) compute(s, stage, !(s + BT <= hi_min && (s >= lo_max || s + BT <= sinks)), copies);
        else if constexpr (decltype(copies)::value) copy_all();
    };
    int stage = 0, b = bfirst;
    for (; b + bstep < b1; b += bstep) {
        block(b, stage, std::true_type{});
        stage ^= 1;
    }
    if (b < b1) block(b, stage, std::false_type{});

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
            const size_t at = row_at * a.all + piece0 + piece;
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
                const size_t at = ra * a.all + piece0 + piece;
                if (b0 < b1) *reinterpret_cast<f32x4_t*>(a.part + at * Dp + d) = acc;
                if (d == 0) a.ml[at] = make_float2(M, L);
            }
        }
    }
}

}  // namespace bitq
