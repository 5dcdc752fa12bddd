// Attention of one new token per request over the paged cache of libbitq.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "bitq_device.h"

namespace bitq {

// out = sum_t p_t V_t / sum_t p_t, p_t = exp(scale q . K_t): every key and
// value is read once and used for the `group` query heads that share it, so
// the kernel is bound by the memory stream.  One pass: each wave keeps a
// running maximum m, sum l and accumulator O per query head, in fp32, and
// rescales O and l when m grows.
//
// Measured (rows of 128): 3 requests of 131072 tokens, 64 heads on 8, bf16,
// 274 us with the join, 5.9 TB/s; 64 ragged requests of up to 8192 tokens,
// int8, 80 + 5 us, 4.6 TB/s (a copy of the kernel that only loads was 6 %
// faster: pages of 32 tokens are 4 KB pieces); one request of 2049 tokens, 32
// heads, 11 + 4 us, of which 7 are its 34 MB and the rest the chain of lengths,
// table, keys and join.
//
// Matrix cores.  A wave takes steps of 32 tokens of one key-value head and a
// tile of 16 query heads:
//   S[32 tokens][16 heads] = K q^T   (two 16-token tiles, A = K rows)
//   O^T[Dp][16 heads] += V^T P       (A = V^T, B = P)
// with v_mfma_f32_16x16x32_bf16: lane l = 16 g + j holds 8 consecutive k of
// row (column) j of A (B), and rows 4 g + i, i < 4, of column j of D.  Row
// 4 g + i of score tile t is given token 8 g + 4 t + i, so that a lane's 8
// scores are those of 8 consecutive tokens 8 g .. 8 g + 7 of head j: exactly
// the B operand that the second product needs from that lane, with no
// movement between lanes.  V's layout (8 tokens of an element together) makes
// its A operand one 16-byte load.  Keys and values go from memory to registers;
// LDS holds the queries' operands and joins the waves at the end.  With fewer
// than 16 query heads per key-value head columns idle: the matrix cores need a
// tenth of the memory's time even so.
//
// Precision.  bf16 and int8 cache rows are exact in bf16; int8 scales are
// applied in fp32, to the scores and to p.  fp32 q is split into 3 bf16
// terms, which hold its 24 bits, bf16 q needs one.  p (times V's scale) is
// split into 3 terms alike: 2 (2^-17) would change the rounding of one bf16
// output in a thousand over a long context and save nothing there (bf16 rows;
// int8, 64 ragged requests of up to 4096 tokens, us with 2 and 3: rows of 64
// 41.7 and 43.5, 128 71.5 and 72.6, 256 123 and 124).  Everything else is
// fp32.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct AttnArgs {
    const void* q;
    const uint8_t* cache;
    const int32_t* table;
    const int32_t* lens;
    void* out;
    float* lse;
    float* part;       // split: partial results, two per workgroup
    int32_t* prefix;   // split: [R + 1] prefix sums of the requests' units
    int64_t q_stride;
    size_t off_v, off_ks, off_vs;
    int R, H, A, group, tiles, D, page_shift, pages, table_stride, max_len, window;
    float c;           // scale log2(e): p = 2^(c s - m)
    int odt;
    int qvec;          // 16-byte loads of q: D a multiple of 8, rows and base aligned
};

// Tokens [lo, hi) of request r.
__device__ __forceinline__ int first_token(const AttnArgs& a, int hi) { return a.window > 0 ? max(hi - a.window, 0) : 0; }
__device__ __forceinline__ void token_range(const AttnArgs& a, int r, int& lo, int& hi) {
    hi = min(max(a.lens[r], 0), a.max_len);
    lo = first_token(a, hi);
}
// Passes of a workgroup over [lo, hi): steps are aligned to 32 tokens.
__device__ __forceinline__ int token_units(int lo, int hi) {
    return hi > lo ? (hi - (lo & ~31) + kAttnUnit - 1) / kAttnUnit : 0;
}

// (2^x by the hardware instruction: 1 ulp, results below 2^-126 flushed to 0)
//
// Maximum / sum over the four lanes 16 g + j of a column.
__device__ __forceinline__ float col_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float col_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// x = sum of the N bf16 terms, each the rounding of what the ones before leave
template <int N>
__device__ __forceinline__ void split_terms(const float (&x)[8], bf16x8_t (&t)[N]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[n][e] = static_cast<__bf16>(r[e]);
            r[e] -= static_cast<float>(t[n][e]);
        }
}

// Place of element d of a query head in the operands of S = K q^T: chunk c,
// lane group g, position e.  bf16 rows: d = 32 c + 8 g + e.  int8 rows: a
// lane's 16-byte load covers two chunks, d = 64 (c / 2) + 16 g + 8 (c % 2) + e
// (a last odd chunk as for bf16).
template <bool I8, int NC>
__device__ __forceinline__ int q_place(int d, int head) {
    const bool pair = I8 && d < 64 * (NC / 2);
    const int c = pair ? 2 * (d >> 6) + ((d >> 3) & 1) : d >> 5;
    const int g = pair ? (d >> 4) & 3 : (d >> 3) & 3;
    return ((c * 64) + 16 * g + head) * 8 + (d & 7);
}

// 8 int8 codes as bf16 (exact)
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t lo, uint32_t hi) {
    bf16x8_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(lo >> (8 * e))));
        v[4 + e] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(hi >> (8 * e))));
    }
    return v;
}

// What a wave reads for one step of 32 tokens, as loaded.
template <int KVT, int NC>
struct AttnStep {
    uint4 k[2][KVT == BITQ_KV_BF16 ? NC : (NC + 1) / 2];
    uint4 v[KVT == BITQ_KV_BF16 ? 2 * NC : NC];
    float4 ks[KVT == BITQ_KV_INT8 ? 2 : 1], vs[KVT == BITQ_KV_INT8 ? 2 : 1];
};

template <int KVT, int NC, bool Q32>
struct AttnWave {
    static constexpr int NQ = Q32 ? 3 : 1, NP = 3, Dp = 32 * NC;
    static constexpr bool I8 = KVT == BITQ_KV_INT8;
    bf16x8_t q[Q32 ? 1 : NC];  // bf16 q: the operands; else they are read from LDS where they are used
    f32x4_t o[2 * NC];
    float m, l;
    const AttnArgs& a;
    const int lane, g, j;
    const __bf16* sq;    // the query tile's operands in LDS: [NQ][NC][64 lanes][8]
    const int32_t* row;  // the request's row of the table
    int h, lo, hi, last;

    __device__ __forceinline__ AttnWave(const AttnArgs& args, int ln, const __bf16* s)
        : a(args), lane(ln), g(ln >> 4), j(ln & 15), sq(s) {}

    __device__ __forceinline__ bf16x8_t q_operand(int n, int c) const {
        return *reinterpret_cast<const bf16x8_t*>(sq + ((n * NC + c) * 64 + lane) * 8);
    }

    __device__ __forceinline__ void range(int r, int hk, int lo_, int hi_) {
        h = hk;
        lo = lo_;
        hi = hi_;
        last = max(hi - 1, 0);  // (an empty request reads what its table's first place names, and uses none of it)
        row = a.table + static_cast<size_t>(r) * a.table_stride;
    }
    __device__ __forceinline__ void begin() {
        if constexpr (!Q32) {
#pragma unroll
            for (int c = 0; c < NC; ++c) q[c] = q_operand(0, c);
        }
#pragma unroll
        for (int c = 0; c < 2 * NC; ++c) o[c] = f32x4_t{0, 0, 0, 0};
        m = -FLT_MAX;
        l = 0.0f;
    }

    // Tokens whose data this lane loads for the step at token s, kept inside
    // [lo, hi) (what lies outside is masked in compute): K rows of the two
    // tiles, V group (and scales).
    __device__ __forceinline__ void tokens(int s, int (&tok)[3]) const {
        const int k = s + 8 * (j >> 2) + (j & 3);
        tok[0] = min(max(k, lo), last);
        tok[1] = min(max(k + 4, lo), last);
        tok[2] = min(max(s + 8 * g, lo & ~7), last & ~7);
    }
    __device__ __forceinline__ void lookup(int s, int (&pg)[3]) const {
        int tok[3];
        tokens(s, tok);
#pragma unroll
        for (int i = 0; i < 3; ++i) pg[i] = row[tok[i] >> a.page_shift];
    }

    // Row of the pool of token tok, whose page is pg.
    __device__ __forceinline__ size_t pool_row(int tok, int pg) const {
        const uint32_t p = static_cast<uint32_t>(pg) < static_cast<uint32_t>(a.pages) ? pg : 0;
        return ((static_cast<size_t>(p) * a.H + h) << a.page_shift) + (tok & ((1 << a.page_shift) - 1));
    }
    __device__ __forceinline__ void load_k(int s, const int (&pg)[3], AttnStep<KVT, NC>& L) const {
        constexpr int es = I8 ? 1 : 2;
        int tok[3];
        tokens(s, tok);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* kp = a.cache + pool_row(tok[t], pg[t]) * (Dp * es);
            if constexpr (!I8) {
                kp += 16 * g;
#pragma unroll
                for (int c = 0; c < NC; ++c) L.k[t][c] = *reinterpret_cast<const uint4*>(kp + 64 * c);
            } else {
#pragma unroll
                for (int c = 0; c < NC / 2; ++c) L.k[t][c] = *reinterpret_cast<const uint4*>(kp + 64 * c + 16 * g);
                if constexpr (NC % 2) {
                    const uint2 u = *reinterpret_cast<const uint2*>(kp + 32 * (NC - 1) + 8 * g);
                    L.k[t][NC / 2] = make_uint4(u.x, u.y, 0, 0);
                }
            }
        }
        if constexpr (I8) {
            const float4* p = reinterpret_cast<const float4*>(a.cache + a.off_ks) + pool_row(tok[2], pg[2]) / 4;
            L.ks[0] = p[0];
            L.ks[1] = p[1];
        }
    }
    __device__ __forceinline__ void load_v(int s, const int (&pg)[3], AttnStep<KVT, NC>& L) const {
        constexpr int es = I8 ? 1 : 2;
        int tok[3];
        tokens(s, tok);
        const size_t at = pool_row(tok[2], pg[2]);  // (a multiple of 8: groups of 8 rows)
        const uint8_t* vp = a.cache + a.off_v + at * (Dp * es) + 16 * j;
        // bf16: 16 bytes are element 16 c + j of 8 tokens; int8: elements 32 c + 2 j and 32 c + 2 j + 1
#pragma unroll
        for (int c = 0; c < (I8 ? NC : 2 * NC); ++c) L.v[c] = *reinterpret_cast<const uint4*>(vp + 256 * c);
        if constexpr (I8) {
            const float4* p = reinterpret_cast<const float4*>(a.cache + a.off_vs) + at / 4;
            L.vs[0] = p[0];
            L.vs[1] = p[1];
        }
    }

    // Scores of tokens s + 8 g + e, scaled to powers of two; masked ones are
    // -inf.  keep: bit e is set if the token is in [lo, hi).
    __device__ __forceinline__ void scores(int s, const AttnStep<KVT, NC>& L, float (&x)[8], uint32_t& keep, bool edge) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                bf16x8_t kf;
                if constexpr (!I8) {
                    kf = __builtin_bit_cast(bf16x8_t, L.k[t][c]);
                } else {
                    const uint4 u = L.k[t][c >> 1];
                    kf = (c & 1) ? codes_bf16(u.z, u.w) : codes_bf16(u.x, u.y);
                }
#pragma unroll
                for (int n = NQ - 1; n >= 0; --n)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, Q32 ? q_operand(n, c) : q[Q32 ? 0 : c], acc, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * t + i] = acc[i];
        }
        if constexpr (I8) {
            const float ks[8] = {L.ks[0].x, L.ks[0].y, L.ks[0].z, L.ks[0].w, L.ks[1].x, L.ks[1].y, L.ks[1].z, L.ks[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= ks[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= a.c;
        keep = 0xFFu;
        if (edge) {
            asm volatile("");  // (a branch, not selects in every step)
            keep = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int tk = s + 8 * g + e;
                const bool in = tk >= lo && tk < hi;
                keep |= in ? 1u << e : 0u;
                x[e] = in ? x[e] : -INFINITY;
            }
        }
    }

    // The weights p of those scores (in x), with m, l and O rescaled if m grows.
    __device__ __forceinline__ void weights(float (&x)[8]) {
        float mx = -FLT_MAX;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, x[e]);
        mx = col_max(mx);
        if (__any(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int c = 0; c < 2 * NC; ++c) o[c] *= f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = __builtin_amdgcn_exp2f(x[e] - m);
            l += x[e];
        }
    }

    __device__ __forceinline__ void values(AttnStep<KVT, NC>& L, float (&p)[8], uint32_t keep, bool edge) {
        if constexpr (I8) {
            float vs[8] = {L.vs[0].x, L.vs[0].y, L.vs[0].z, L.vs[0].w, L.vs[1].x, L.vs[1].y, L.vs[1].z, L.vs[1].w};
            if (edge) {  // scales in masked places may be infinite or NaN
                asm volatile("");
#pragma unroll
                for (int e = 0; e < 8; ++e) vs[e] = keep & (1u << e) ? vs[e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] *= vs[e];
        }
        bf16x8_t pf[NP];
        split_terms<NP>(p, pf);
        if (!I8 && edge) {  // what lies in masked places may be infinite or NaN: 0 p must stay 0
            asm volatile("");
            uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 1] &= keep & (1u << e) ? ~0u : (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
            for (int c = 0; c < 2 * NC; ++c) {
                uint4& u = L.v[I8 ? 0 : c];
                u = make_uint4(u.x & w[0], u.y & w[1], u.z & w[2], u.w & w[3]);
            }
        }
#pragma unroll
        for (int c = 0; c < 2 * NC; ++c) {
            bf16x8_t vf;
            if constexpr (!I8) {
                vf = __builtin_bit_cast(bf16x8_t, L.v[c]);
            } else {
                const uint4 u = L.v[c >> 1];  // (int8 codes are finite whatever the bytes)
                vf = (c & 1) ? codes_bf16(u.z, u.w) : codes_bf16(u.x, u.y);
            }
#pragma unroll
            for (int n = NP - 1; n >= 0; --n)
                o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[n], o[c], 0, 0, 0);
        }
    }

    // The wave's steps s0, s0 + stride, ... below s1.  A step's registers are
    // loaded again as soon as they are free: the next keys are in flight
    // while the weights and values are worked on, the next values while the
    // next scores are.  The last step, which loads nothing, is code of its
    // own: behind a branch in the loop the compiler would wait for all loads.
    // (A second set of registers measured no better.)
    template <bool LAST>
    __device__ __forceinline__ void step(int s, int next, int after, AttnStep<KVT, NC>& L, int (&pg)[3]) {
        const bool edge = s < lo || s + 32 > hi;  // (the same for the whole wave)
        float x[8];
        uint32_t keep;
        asm volatile("" ::: "memory");  // (q's operands are read again, not kept in registers)
        scores(s, L, x, keep, edge);
        if constexpr (!LAST) load_k(next, pg, L);
        weights(x);
        values(L, x, keep, edge);
        if constexpr (!LAST) {
            load_v(next, pg, L);
            lookup(after, pg);
        }
    }
    __device__ __forceinline__ void first(int s0, int s1, int stride, AttnStep<KVT, NC>& L, int (&pg)[3]) {
        lookup(s0, pg);
        load_k(s0, pg, L);
        load_v(s0, pg, L);
        if (s0 + stride < s1) lookup(s0 + stride, pg);
    }
    __device__ __forceinline__ void run(int s0, int s1, int stride, AttnStep<KVT, NC>& L, int (&pg)[3]) {
        if (s0 >= s1) return;
        int s = s0;
        for (; s + stride < s1; s += stride) step<false>(s, s + stride, min(s + 2 * stride, last), L, pg);
        step<true>(s, 0, 0, L, pg);
    }

    // O, m, l to the wave's part of LDS: so [16][Dp + 4], sm and sl [16].
    __device__ __forceinline__ void park(float* so, float* sm, float* sl) {
        l = col_sum(l);
        if (g == 0) {
            sm[j] = m;
            sl[j] = l;
        }
        float* r = so + j * (Dp + 4);
        if constexpr (!I8) {
#pragma unroll
            for (int c = 0; c < 2 * NC; ++c) *reinterpret_cast<f32x4_t*>(r + 16 * c + 4 * g) = o[c];
        } else {
            // tile 2c + b, row 4 g + i is element 32 c + 2 (4 g + i) + b
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const f32x4_t u = o[2 * c], w = o[2 * c + 1];
                *reinterpret_cast<f32x4_t*>(r + 32 * c + 8 * g) = f32x4_t{u[0], w[0], u[1], w[1]};
                *reinterpret_cast<f32x4_t*>(r + 32 * c + 8 * g + 4) = f32x4_t{u[2], w[2], u[3], w[3]};
            }
        }
    }
};

__device__ __forceinline__ void store_out(const AttnArgs& a, size_t i, float v) {
    if (a.odt == BITQ_DT_F32) static_cast<float*>(a.out)[i] = v;
    else static_cast<uint16_t*>(a.out)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Sum over lanes 0 .. this lane.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1, 2, 4 and 8 lanes below, in a row of 16
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of a row to the row above: rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
    return v;
}

// The deal of T units to G workgroups (at most 1024): workgroup i has units
// [start(i), start(i + 1)), start(i) = floor(T i / G).  With T = q G + rem it is
// i q + floor(rem i / G), and rem i < 2^20, so the fp32 quotient of rem i +
// 1/2 is off by less than 1/(2 G) and rounds down to the right integer.
struct AttnRanges {
    uint32_t T, G, q, rem;
    float inv;
    __device__ __forceinline__ AttnRanges(uint32_t units, uint32_t grid) : T(units), G(min(units, grid)) {
        q = T / max(G, 1u);
        rem = T - q * G;
        inv = 1.0f / static_cast<float>(G);
    }
    __device__ __forceinline__ uint32_t start(uint32_t i) const {
        return i * q + static_cast<uint32_t>((static_cast<float>(rem * i) + 0.5f) * inv);
    }
    // the workgroup that has unit x < T
    __device__ __forceinline__ uint32_t owner(uint32_t x) const {
        uint32_t i = min(static_cast<uint32_t>(static_cast<float>(x) * (static_cast<float>(G) / static_cast<float>(T))), G - 1);
        while (start(i) > x) --i;
        while (start(i + 1) <= x) ++i;
        return i;
    }
};

// First index i in [0, n) with a[i] > x (n if none); a ascending.
__device__ __forceinline__ int first_above32(const int32_t* a, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// SPLIT = false: workgroup = one item (request, key-value head, tile of 16 of
// its query heads), its tokens dealt to the waves in steps of 32.
// SPLIT = true: the items' tokens, in units of 128, are laid end to end (head
// tiles outermost, then requests) and dealt to the gridDim.x workgroups in
// equal contiguous ranges, so ragged lengths load every workgroup alike.
// A range that covers an item whole writes its output; the ends of an item
// that lies in several ranges go to the workgroup's two partial results (slot
// 0: an item begun elsewhere, slot 1: one begun here) for the join kernel.
template <int KVT, int NC, bool Q32, bool SPLIT, int W>
__global__ __launch_bounds__(64 * W, attn_groups_per_cu(KVT, NC, Q32) * kAttnWaves / W) void paged_attn_kernel(AttnArgs a) {
    constexpr int Dp = 32 * NC, ROW = Dp + 4;
    static_assert(!SPLIT || W == kAttnWaves, "a unit is a pass of kAttnWaves waves");
    __shared__ __align__(16) float s_o[W][16 * ROW];
    __shared__ float s_m[W][16], s_l[W][16];
    constexpr int NQ = Q32 ? 3 : 1, QP = (2 * Dp + 64 * W - 1) / (64 * W);
    __shared__ __align__(16) __bf16 s_q[NQ * 16 * Dp];
    extern __shared__ int32_t s_pre[];  // SPLIT: [R + 1]
    __shared__ int32_t s_scan[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int HT = a.H * a.tiles;
    AttnWave<KVT, NC, Q32> w(a, lane, s_q);

    int x = blockIdx.x, x1 = x + 1;  // units (SPLIT; fewer than 2^31) or the item
    int U = 1;
    // up to 64 requests: lane r of every wave keeps request r's length and
    // the end of its units, and a unit's request is found by one vote; more:
    // the prefix sums are in LDS and searched (lens read again)
    const bool few = a.R <= 64;
    int my_hi = 0, my_end = 0;
    if constexpr (SPLIT) {
        if (few) {
            int lo = 0;
            if (lane < a.R) token_range(a, lane, lo, my_hi);
            my_end = wave_scan(token_units(lo, my_hi));
            U = __builtin_amdgcn_readlane(my_end, 63);
            if (blockIdx.x == 0 && wave == 0) {
                if (lane < a.R) a.prefix[lane + 1] = my_end;
                if (lane == 0) a.prefix[0] = 0;
            }
        } else {
            int carry = 0;
            for (int r0 = 0; r0 < a.R; r0 += 64 * W) {
                const int r = r0 + tid;
                int lo = 0, hi = 0;
                if (r < a.R) token_range(a, r, lo, hi);
                int inc = wave_scan(token_units(lo, hi));
                __syncthreads();
                if (lane == 63) s_scan[wave] = inc;
                __syncthreads();
                int all = 0;
                for (int i = 0; i < W; ++i) {
                    if (i < wave) inc += s_scan[i];
                    all += s_scan[i];
                }
                if (r < a.R) s_pre[r + 1] = carry + inc;
                carry += all;
            }
            if (tid == 0) s_pre[0] = 0;
            __syncthreads();
            if (blockIdx.x == 0)
                for (int r = tid; r <= a.R; r += 64 * W) a.prefix[r] = s_pre[r];
            U = wave_uniform(s_pre[a.R]);
        }
        const uint32_t T = static_cast<uint32_t>(U) * HT;  // (< 2^31)
        // (with fewer units than workgroups the surplus workgroups have none:
        // every range below G is non-empty, which the join relies on)
        const AttnRanges ranges(T, gridDim.x);
        if (blockIdx.x >= ranges.G) return;
        x = ranges.start(blockIdx.x);
        x1 = ranges.start(blockIdx.x + 1);
    }
    while (x < x1) {
        int ht, r, lo, hi, s0, s1;
        bool whole = true;
        int slot = 0, next = x + 1;
        if constexpr (SPLIT) {
            ht = static_cast<uint32_t>(x) / static_cast<uint32_t>(U);
            const int rem = x - ht * U;
            int begin, end;  // of the request's units
            if (few) {
                r = __builtin_ctzll(__ballot(my_end > rem));  // (rem < U = the last lane's)
                hi = __builtin_amdgcn_readlane(my_hi, r);
                lo = first_token(a, hi);
                end = __builtin_amdgcn_readlane(my_end, r);
                begin = r > 0 ? __builtin_amdgcn_readlane(my_end, r - 1) : 0;
            } else {
                r = wave_uniform(first_above32(s_pre + 1, a.R, rem));
                token_range(a, r, lo, hi);
                begin = wave_uniform(s_pre[r]);
                end = wave_uniform(s_pre[r + 1]);
            }
            end += ht * U;
            next = min(x1, end);
            const int k0 = rem - begin;
            whole = k0 == 0 && next == end;
            slot = k0 == 0 ? 1 : 0;
            s0 = (lo & ~31) + k0 * kAttnUnit;
            s1 = min(hi, s0 + (next - x) * kAttnUnit);
        } else {
            ht = x % HT;
            r = x / HT;
            token_range(a, r, lo, hi);
            s0 = lo & ~31;
            s1 = hi;
        }
        // (values that are the same for the whole wave, kept in scalar registers)
        const int hk = static_cast<uint32_t>(ht) / static_cast<uint32_t>(a.tiles), tile = ht - hk * a.tiles;
        const int heads = min(16, a.group - 16 * tile);
        // ---- the tile's queries, 8 elements of a head at a time; then the first step's loads, behind them
        const int64_t qat = static_cast<int64_t>(r) * a.q_stride + (static_cast<int64_t>(hk) * a.group + 16 * tile) * a.D;
        uint32_t qv[QP][8];
#pragma unroll
        for (int u = 0; u < QP; ++u) {
            const int i = tid + 64 * W * u, head = min(i / (Dp / 8), heads - 1), d = 8 * (i % (Dp / 8));
            // (as loaded: a conversion here would wait for the loads)
            if (a.qvec) {
                const uint8_t* p = static_cast<const uint8_t*>(a.q) + (qat + head * a.D + min(d, a.D - 8)) * (Q32 ? 4 : 2);
                const uint4 v0 = reinterpret_cast<const uint4*>(p)[0];
                qv[u][0] = v0.x, qv[u][1] = v0.y, qv[u][2] = v0.z, qv[u][3] = v0.w;
                if (Q32) {
                    const uint4 v1 = reinterpret_cast<const uint4*>(p)[1];
                    qv[u][4] = v1.x, qv[u][5] = v1.y, qv[u][6] = v1.z, qv[u][7] = v1.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t at = head * a.D + min(d + e, a.D - 1);
                    if (Q32) qv[u][e] = (static_cast<const uint32_t*>(a.q) + qat)[at];
                    else qv[u][e] = (static_cast<const uint16_t*>(a.q) + qat)[at];
                }
            }
        }
        AttnStep<KVT, NC> L;
        int pg[3];
        const int from = wave_uniform(s0) + 32 * wave, upto = wave_uniform(s1);
        w.range(r, hk, wave_uniform(lo), wave_uniform(hi));
        w.first(from, upto, 32 * W, L, pg);
        // ---- into LDS as the terms and in the order of the operands
#pragma unroll
        for (int u = 0; u < QP; ++u) {
            const int i = tid + 64 * W * u, head = i / (Dp / 8), d = 8 * (i % (Dp / 8));
            if (i >= 2 * Dp) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t pair = qv[u][e / 2];
                const uint32_t bits = Q32 ? qv[u][e] : !a.qvec ? qv[u][e] << 16 : e & 1 ? pair & 0xFFFF0000u : pair << 16;
                f[e] = head < heads && d + e < a.D ? __uint_as_float(bits) : 0.0f;
            }
            bf16x8_t t[NQ];
            split_terms<NQ>(f, t);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                *reinterpret_cast<bf16x8_t*>(s_q + n * (16 * Dp) + q_place<KVT == BITQ_KV_INT8, NC>(d, head)) = t[n];
        }
        __syncthreads();
        w.begin();
        w.run(from, upto, 32 * W, L, pg);
        w.park(s_o[wave], s_m[wave], s_l[wave]);
        __syncthreads();
        float* part = SPLIT ? a.part + (static_cast<size_t>(blockIdx.x) * 2 + slot) * (16 * (Dp + 2)) : nullptr;
        for (int i = tid; i < heads * Dp; i += 64 * W) {
            const int head = i / Dp, d = i - head * Dp;
            float M = s_m[0][head];
#pragma unroll
            for (int v = 1; v < W; ++v) M = fmaxf(M, s_m[v][head]);
            float sum = 0.0f, acc = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const float f = __builtin_amdgcn_exp2f(s_m[v][head] - M);
                sum += f * s_l[v][head];
                acc += f * s_o[v][head * ROW + d];
            }
            if (whole) {
                const size_t qa = static_cast<size_t>(r) * a.A + static_cast<size_t>(hk) * a.group + 16 * tile + head;
                if (d < a.D) store_out(a, qa * a.D + d, sum == 0.0f ? 0.0f : acc / sum);
                if (d == 0 && a.lse) a.lse[qa] = lse_of(M, sum);
            } else {
                part[head * Dp + d] = acc;
                if (d == 0) {
                    part[16 * Dp + head] = M;
                    part[16 * Dp + 16 + head] = sum;
                }
            }
        }
        __syncthreads();
        x = next;
    }
}

// Maximum / sum over the wave: in the last lane by the steps of wave_scan, then in all.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float v, float none) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(none), __float_as_uint(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float join_max(float v) {  // (v >= -FLT_MAX)
    v = fmaxf(v, dpp_or<0x111, 0xf>(v, -FLT_MAX));
    v = fmaxf(v, dpp_or<0x112, 0xf>(v, -FLT_MAX));
    v = fmaxf(v, dpp_or<0x114, 0xf>(v, -FLT_MAX));
    v = fmaxf(v, dpp_or<0x118, 0xf>(v, -FLT_MAX));
    v = fmaxf(v, dpp_or<0x142, 0xa>(v, -FLT_MAX));
    v = fmaxf(v, dpp_or<0x143, 0xc>(v, -FLT_MAX));
    return last_lane(v);
}
__device__ __forceinline__ float join_sum(float v) {
    v += dpp_or<0x111, 0xf>(v, 0.0f);
    v += dpp_or<0x112, 0xf>(v, 0.0f);
    v += dpp_or<0x114, 0xf>(v, 0.0f);
    v += dpp_or<0x118, 0xf>(v, 0.0f);
    v += dpp_or<0x142, 0xa>(v, 0.0f);
    v += dpp_or<0x143, 0xc>(v, 0.0f);
    return last_lane(v);
}

// Joins the partial results of the items that lie in several workgroups'
// ranges, and writes the outputs of requests without tokens.  NW waves per
// query head: one when there are many heads (4 heads a workgroup), 8 or 16
// when there are few and an item may lie in hundreds of ranges.  Bound by
// latency: m and l of 64 partial results are loaded at once, a lane each, and
// with them the first rows of the accumulators (Dp <= 64 NE floats); further
// rows are loaded four at a time with their weights 2^(m - M) known, so the
// loads do not wait for each other.  (A chain of one partial result after the
// other took 17.5 us instead of 8.4 for 8 heads of 512 ranges.)
template <int NW, int NE>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void attn_join_kernel(AttnArgs a, int Dp, int main_grid) {
    constexpr int HPB = NW == 1 ? 4 : 1, AHEAD = 4;
    __shared__ float s_acc[NW][64 * NE], s_m[NW], s_l[NW];
    const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
    const uint32_t qa = blockIdx.x * HPB + (NW == 1 ? wave : 0);
    if (qa >= static_cast<uint32_t>(a.R) * a.A) return;
    const int r = qa / static_cast<uint32_t>(a.A), qh = qa - r * a.A;
    const int hk = static_cast<uint32_t>(qh) / static_cast<uint32_t>(a.group), in = qh - hk * a.group;
    const int ht = hk * a.tiles + (in >> 4), head = in & 15;
    const int U = a.prefix[a.R], u0 = a.prefix[r], u1 = a.prefix[r + 1];
    float acc[NE] = {}, M = -FLT_MAX, L = 0.0f;
    if (u1 > u0) {
        const AttnRanges ranges(U * a.H * a.tiles, main_grid);
        const int i0 = ranges.owner(ht * U + u0), i1 = ranges.owner(ht * U + u1 - 1);
        if (i0 == i1) return;  // whole in one range: written there
        const uint32_t size = 16 * (Dp + 2);
        auto part = [&](int i) { return a.part + (static_cast<uint32_t>(i) * 2 + (i == i0 ? 1 : 0)) * size; };
        const int per = (i1 - i0 + NW) / NW, from = i0 + (NW == 1 ? 0 : wave * per), to = min(i1 + 1, from + per);
        for (int c = from; c < to; c += 64) {
            const int n = min(64, to - c);
            const float* p = part(min(c + lane, to - 1)) + 16 * Dp + head;
            float pm = p[0], pl = p[16], v[AHEAD][NE];
            auto rows = [&](int j) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < AHEAD; ++q) {
                    const float* row = part(c + min(j + q, n - 1)) + head * Dp;
#pragma unroll
                    for (int e = 0; e < NE; ++e) v[q][e] = row[min(lane + 64 * e, Dp - 1)];
                }
            };
            rows(0);
            pm = lane < n ? pm : -FLT_MAX;
            const float mn = fmaxf(M, join_max(pm)), f = __builtin_amdgcn_exp2f(M - mn), w = __builtin_amdgcn_exp2f(pm - mn);
            M = mn;
            L = L * f + join_sum(lane < n ? pl * w : 0.0f);
#pragma unroll
            for (int e = 0; e < NE; ++e) acc[e] *= f;
            for (int j = 0; j < n; j += AHEAD) {
                if (j > 0) rows(j);
#pragma unroll
                for (int q = 0; q < AHEAD; ++q) {
                    const float wq = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), min(j + q, n - 1)));
#pragma unroll
                    for (int e = 0; e < NE; ++e) acc[e] += j + q < n ? v[q][e] * wq : 0.0f;
                }
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
        if (d < a.D) store_out(a, static_cast<size_t>(qa) * a.D + d, L == 0.0f ? 0.0f : acc[e] / L);
    }
    if (lane == 0 && a.lse) a.lse[qa] = lse_of(M, L);
}

// Waves per query head, measured in us: 32 heads of 17 ranges each 4.0 with 8
// and 4.6 with 16; 8 heads of 512 ranges 11.4 and 8.4; 640
// heads of a few 4.7 with 1.
template <int NE>
static void launch_join(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const unsigned heads = static_cast<unsigned>(a.R) * a.A;
    if (heads > 512)
        hipLaunchKernelGGL((attn_join_kernel<1, NE>), dim3((heads + 3) / 4), dim3(256), 0, st, a, p.Dp, p.grid);
    else if (p.grid / p.items < 64)
        hipLaunchKernelGGL((attn_join_kernel<8, NE>), dim3(heads), dim3(512), 0, st, a, p.Dp, p.grid);
    else
        hipLaunchKernelGGL((attn_join_kernel<16, NE>), dim3(heads), dim3(1024), 0, st, a, p.Dp, p.grid);
}

template <int KVT, int NC, bool Q32>
static void launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(p.grid)), block(64 * p.waves);
    if (!p.split) {
        if (p.waves == 1) hipLaunchKernelGGL((paged_attn_kernel<KVT, NC, Q32, false, 1>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((paged_attn_kernel<KVT, NC, Q32, false, kAttnWaves>), grid, block, 0, st, a);
        return;
    }
    hipLaunchKernelGGL((paged_attn_kernel<KVT, NC, Q32, true, kAttnWaves>), grid, block, 4 * (static_cast<size_t>(a.R) + 1), st, a);
    launch_join<(NC + 1) / 2>(a, p, st);
}

template <int KVT, bool Q32>
static void launch_attn_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    switch (p.Dp / 32) {
        case 1: launch_attn<KVT, 1, Q32>(a, p, st); break;
        case 2: launch_attn<KVT, 2, Q32>(a, p, st); break;
        case 3: launch_attn<KVT, 3, Q32>(a, p, st); break;
        case 4: launch_attn<KVT, 4, Q32>(a, p, st); break;
        case 5: launch_attn<KVT, 5, Q32>(a, p, st); break;
        case 6: launch_attn<KVT, 6, Q32>(a, p, st); break;
        case 7: launch_attn<KVT, 7, Q32>(a, p, st); break;
        default: launch_attn<KVT, 8, Q32>(a, p, st); break;
    }
}

int launch_paged_attn(const bitq_attn_desc& d, const AttnPlan& plan, const void* q, int64_t q_stride,
                      const void* cache, const int32_t* table, const int32_t* lens, void* out, float* lse, void* ws,
                      void* stream) {
    const KvLayout L = kv_layout(d.kv);
    AttnArgs a{};
    a.q = q;
    a.cache = static_cast<const uint8_t*>(cache);
    a.table = table;
    a.lens = lens;
    a.out = out;
    a.lse = lse;
    a.prefix = static_cast<int32_t*>(ws);
    a.part = plan.split ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan.off_part) : nullptr;
    a.q_stride = q_stride;
    a.off_v = L.off_v;
    a.off_ks = L.off_ks;
    a.off_vs = L.off_vs;
    a.R = d.requests;
    a.H = d.kv.kv_heads;
    a.A = d.heads;
    a.group = plan.group;
    a.tiles = plan.tiles;
    a.D = d.kv.head_dim;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(d.kv.page));
    a.pages = d.kv.pages;
    a.table_stride = d.table_stride;
    a.max_len = d.max_len;
    a.window = d.window;
    a.c = d.scale * 1.44269504088896340736f;
    a.odt = d.out_dtype;
    const int per16 = d.q_dtype == BITQ_DT_F32 ? 4 : 8;
    a.qvec = a.D % 8 == 0 && q_stride % per16 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool q32 = d.q_dtype == BITQ_DT_F32;
    if (d.kv.dtype == BITQ_KV_BF16) {
        if (q32) launch_attn_dim<BITQ_KV_BF16, true>(a, plan, st);
        else launch_attn_dim<BITQ_KV_BF16, false>(a, plan, st);
    } else {
        if (q32) launch_attn_dim<BITQ_KV_INT8, true>(a, plan, st);
        else launch_attn_dim<BITQ_KV_INT8, false>(a, plan, st);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
