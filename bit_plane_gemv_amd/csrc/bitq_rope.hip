// Queries and keys of new tokens: the norm of each head and its rotation by
// position, in one pass over the data.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitq_device.h"

namespace bitq {

// A unit is 16 elements of a head in two parts of 8: the 8 pairs of a
// rotation (halves: elements 8 u .. of each half; neighbours: 16 in a row) or
// 16 elements past the rotated ones.  A lane takes one unit of a head, LPH
// lanes (a power of two) a head, so the two parts are 16-byte loads of bf16
// and the norm is a sum over LPH neighbouring lanes.  The angles depend on the
// token and the unit alone: a lane computes its 8 sines and cosines once and
// keeps them for the heads that it goes through (`passes` of them).
//
// Angles.  table holds each pair's turns per position as a fraction of 2^64;
// position * entry mod 2^64 is the angle with no error beyond the entry's own
// (below 2^-62 turns per position), wherever the position.  Its upper 32 bits are
// cut into a quarter and a rest of at most an eighth of a turn, on which the
// Taylor series of sine (to x^9) and cosine (to x^10) err by less than 2^-28.
// An fp32 angle would be off by up to 0.004 at position 131072.
//
// The sum of squares is over at most 256 elements, in fp32; outputs are rounded once.
//
// Bound by HBM for prompts (each element read and written once): 4096 tokens x
// 72 heads of 128, bf16, half of each head rotated, 36.7 us, 4.1 TB/s; by
// latency for a decode step: 64 tokens, 4.9 us.
struct RopeArgs {
    const void *q, *k, *qw, *kw;
    const uint64_t* table;
    const int32_t* pos;
    void *qo, *ko;
    int64_t qs, ks, qos, kos;
    int T, QH, KH, D, rot, rot_units, units, lph_shift, passes, wdt;
    int q_groups, k_groups;  // lane groups' passes per token
    bool wvec, tvec;         // weights, table: 16-byte aligned
    float eps, mscale, inv_d;
};

// sin and cos of t / 2^32 turns
__device__ __forceinline__ void sincos_turns(uint32_t t, float& s, float& c) {
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(t - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float z = x * x;
    const float sn = x + x * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
    const float cs = 1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320 + z * (-1.0f / 3628800)))));
    s = quarter & 1 ? cs : sn;
    c = quarter & 1 ? sn : cs;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

// elements at .. at + 7 of x, the first n present (VEC: 8 or none, 16-byte aligned)
template <int DT, bool VEC>
__device__ __forceinline__ void rope_load(const void* x, int64_t at, int n, float (&v)[8]) {
    if constexpr (VEC) {
        if (n > 0) {
            const uint8_t* p = static_cast<const uint8_t*>(x) + at * (DT == BITQ_DT_F32 ? 4 : 2);
            const uint4 a = reinterpret_cast<const uint4*>(p)[0];
            if constexpr (DT == BITQ_DT_F32) {
                const uint4 b = reinterpret_cast<const uint4*>(p)[1];
                const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
            } else {
                const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(e & 1 ? u[e >> 1] & 0xFFFF0000u : u[e >> 1] << 16);
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? act_at<DT>(x, at + e) : 0.0f;
    }
}
__device__ __forceinline__ uint32_t rope_bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
template <int DT, bool VEC>
__device__ __forceinline__ void rope_store(void* x, int64_t at, int n, const float (&v)[8]) {
    if (n <= 0) return;
    if constexpr (VEC) {
        uint8_t* p = static_cast<uint8_t*>(x) + at * (DT == BITQ_DT_F32 ? 4 : 2);
        if constexpr (DT == BITQ_DT_F32) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = rope_bits(v[2 * e]) | (rope_bits(v[2 * e + 1]) << 16);
            *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < n) {
                if constexpr (DT == BITQ_DT_F32) static_cast<float*>(x)[at + e] = v[e];
                else static_cast<uint16_t*>(x)[at + e] = static_cast<uint16_t>(rope_bits(v[e]));
            }
        }
    }
}

// Work item = (token, group): 64 / LPH heads at a time for `passes` passes; a
// wave takes one item, q's groups of a token first, then k's.
template <int XDT, int ODT, bool PAIRS, bool VEC>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a) {
    const int lane = threadIdx.x & 63;
    const uint32_t item = blockIdx.x * 4u + static_cast<uint32_t>(wave_uniform(threadIdx.x >> 6));
    const uint32_t per = a.q_groups + a.k_groups;
    const uint32_t t = item / per;
    if (t >= static_cast<uint32_t>(a.T)) return;
    const int pos = a.pos[t];
    if (pos < 0) return;
    int grp = static_cast<int>(item - t * per);
    const bool is_q = grp < a.q_groups;
    if (!is_q) grp -= a.q_groups;
    const int heads = is_q ? a.QH : a.KH;
    const void* x = is_q ? a.q : a.k;
    const void* w = is_q ? a.qw : a.kw;
    void* o = is_q ? a.qo : a.ko;
    const int64_t xrow = static_cast<int64_t>(t) * (is_q ? a.qs : a.ks), orow = static_cast<int64_t>(t) * (is_q ? a.qos : a.kos);
    const int u = lane & ((1 << a.lph_shift) - 1), hpw = 64 >> a.lph_shift;
    const bool turns = u < a.rot_units;
    // elements of the unit's two parts
    int ea, eb, na, nb;
    const int half = a.rot >> 1;
    if (turns && !PAIRS) {
        ea = 8 * u;
        eb = half + 8 * u;
        na = nb = min(8, half - 8 * u);
    } else {
        const int end = turns ? a.rot : a.D;
        ea = turns ? 16 * u : a.rot + 16 * (u - a.rot_units);
        eb = ea + 8;
        na = min(8, end - ea);
        nb = min(8, end - eb);
    }
    if (u >= a.units) na = nb = 0;

    const int h0 = grp * hpw * a.passes + (lane >> a.lph_shift);
    float va[8], vb[8], wa[8], wb[8];
    // (the first head's data and the weights are on their way while the angles are computed)
    const bool live0 = h0 < heads;
    rope_load<XDT, VEC>(x, xrow + static_cast<int64_t>(h0) * a.D + ea, live0 ? na : 0, va);
    rope_load<XDT, VEC>(x, xrow + static_cast<int64_t>(h0) * a.D + eb, live0 ? nb : 0, vb);
    if (w) {
        if (VEC && a.wvec) {
            if (a.wdt == BITQ_DT_F32) {
                rope_load<BITQ_DT_F32, VEC>(w, ea, na, wa);
                rope_load<BITQ_DT_F32, VEC>(w, eb, nb, wb);
            } else {
                rope_load<BITQ_DT_BF16, VEC>(w, ea, na, wa);
                rope_load<BITQ_DT_BF16, VEC>(w, eb, nb, wb);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                wa[e] = e < na ? load_act(w, a.wdt, ea + e) : 0.0f;
                wb[e] = e < nb ? load_act(w, a.wdt, eb + e) : 0.0f;
            }
        }
    }
    float sn[8], cs[8];
    if (turns) {
        const int pairs = PAIRS ? half - 8 * u : na;
        uint64_t fs[8];
        if (VEC && a.tvec && pairs >= 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const ulonglong2 v = reinterpret_cast<const ulonglong2*>(a.table + 8 * u)[e];
                fs[2 * e] = v.x;
                fs[2 * e + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) fs[e] = a.table[8 * u + min(e, pairs - 1)];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t f = fs[e];
            sincos_turns(static_cast<uint32_t>((f * static_cast<uint64_t>(static_cast<uint32_t>(pos))) >> 32), sn[e], cs[e]);
            sn[e] *= a.mscale;
            cs[e] *= a.mscale;
        }
    }
    for (int p = 0; p < a.passes; ++p) {
        const int h = h0 + p * hpw;
        if (wave_uniform(h0 - (lane >> a.lph_shift)) + p * hpw >= heads) break;
        const bool live = h < heads;
        float xa[8], xb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            xa[e] = va[e];
            xb[e] = vb[e];
        }
        if (p + 1 < a.passes) {  // the next head's data
            const int hn = h + hpw;
            rope_load<XDT, VEC>(x, xrow + static_cast<int64_t>(hn) * a.D + ea, hn < heads ? na : 0, va);
            rope_load<XDT, VEC>(x, xrow + static_cast<int64_t>(hn) * a.D + eb, hn < heads ? nb : 0, vb);
        }
        if (w) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += xa[e] * xa[e] + xb[e] * xb[e];
            for (int off = 1; off < (1 << a.lph_shift); off <<= 1) sum += __shfl_xor(sum, off, 64);
            const float r = 1.0f / sqrtf(sum * a.inv_d + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xa[e] = xa[e] * r * wa[e];
                xb[e] = xb[e] * r * wb[e];
            }
        }
        if (turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (PAIRS) {
                    float& u0 = e < 4 ? xa[2 * (e & 3)] : xb[2 * (e & 3)];
                    float& u1 = e < 4 ? xa[2 * (e & 3) + 1] : xb[2 * (e & 3) + 1];
                    const float y0 = u0 * cs[e] - u1 * sn[e], y1 = u1 * cs[e] + u0 * sn[e];
                    u0 = y0;
                    u1 = y1;
                } else {
                    const float y0 = xa[e] * cs[e] - xb[e] * sn[e], y1 = xb[e] * cs[e] + xa[e] * sn[e];
                    xa[e] = y0;
                    xb[e] = y1;
                }
            }
        }
        if (live) {
            rope_store<ODT, VEC>(o, orow + static_cast<int64_t>(h) * a.D + ea, na, xa);
            rope_store<ODT, VEC>(o, orow + static_cast<int64_t>(h) * a.D + eb, nb, xb);
        }
    }
}

template <int XDT, int ODT, bool PAIRS>
static void launch_rope(const RopeArgs& a, bool vec, dim3 grid, hipStream_t st) {
    if (vec) hipLaunchKernelGGL((qk_rope_kernel<XDT, ODT, PAIRS, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((qk_rope_kernel<XDT, ODT, PAIRS, false>), grid, dim3(256), 0, st, a);
}
template <int XDT, int ODT>
static void launch_rope_layout(const RopeArgs& a, bool pairs, bool vec, dim3 grid, hipStream_t st) {
    if (pairs) launch_rope<XDT, ODT, true>(a, vec, grid, st);
    else launch_rope<XDT, ODT, false>(a, vec, grid, st);
}

int launch_qk_rope(const bitq_rope_desc& d, const RopeRows (&rows)[4], const void* qw, const void* kw,
                   const uint64_t* table, const int32_t* pos, void* stream) {
    RopeArgs a{};
    a.q = rows[0].at, a.k = rows[1].at, a.qw = qw, a.kw = kw, a.table = table, a.pos = pos;
    a.qo = const_cast<void*>(rows[2].at), a.ko = const_cast<void*>(rows[3].at);
    a.qs = rows[0].stride, a.ks = rows[1].stride, a.qos = rows[2].stride, a.kos = rows[3].stride;
    a.T = d.tokens, a.QH = d.q_heads, a.KH = d.k_heads, a.D = d.head_dim, a.rot = d.rot, a.wdt = d.w_dtype;
    a.eps = d.eps, a.mscale = d.mscale, a.inv_d = 1.0f / static_cast<float>(d.head_dim);
    a.rot_units = (d.rot / 2 + 7) / 8;
    a.units = a.rot_units + (d.head_dim - d.rot + 15) / 16;
    a.lph_shift = 0;
    while ((1 << a.lph_shift) < a.units) ++a.lph_shift;
    const int hpw = 64 >> a.lph_shift;
    // One pass while the GPU (1024 SIMDs, 5 of these waves each) holds nearly all waves at once; then two heads a lane share its
    // angles.  us in a graph with 1 / 2 passes: 2304 waves (256 tokens x 72 heads of 128, bf16) 5.5 / 6.1, 2560 (512 x 40 of 128,
    // fp32) 6.6 / 7.0, 4096 (1024 x 64 of 64, bf16) 6.8 / 6.5, 4608 (512 x 72) 7.8 / 7.6, 9216 13.0 / 11.7, 36864 38.8 / 31.9;
    // 4 and 8 passes of 36864 took 7 % longer than 2.
    const int64_t waves = static_cast<int64_t>(d.tokens) * ((d.q_heads + hpw - 1) / hpw + (d.k_heads + hpw - 1) / hpw);
    a.passes = waves >= 4096 ? 2 : 1;
    auto groups = [&](int heads) { return (heads + hpw * a.passes - 1) / (hpw * a.passes); };
    auto items_of = [&] { return static_cast<int64_t>(d.tokens) * (groups(d.q_heads) + groups(d.k_heads)); };
    while (items_of() > (int64_t(1) << 25) && a.passes < 16) a.passes *= 2;  // (a launch has fewer than 2^32 threads)
    a.q_groups = groups(d.q_heads);
    a.k_groups = groups(d.k_heads);
    const int64_t items = items_of();
    const dim3 grid(static_cast<unsigned>((items + 3) / 4));
    // parts of 8 elements, all of them whole and 16-byte aligned
    const int es = d.x_dtype == BITQ_DT_F32 ? 4 : 2, eo = d.out_dtype == BITQ_DT_F32 ? 4 : 2;
    const bool pairs = d.layout == BITQ_ROPE_PAIRS;
    bool vec = d.head_dim % 8 == 0 && d.rot % (pairs ? 8 : 16) == 0;
    for (int i = 0; i < 4; ++i)
        vec = vec && (!rows[i].heads || (aligned(rows[i].at, 16) && rows[i].stride % (16 / (i < 2 ? es : eo)) == 0));
    a.wvec = aligned(qw, 16) && aligned(kw, 16);
    a.tvec = aligned(table, 16);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (d.x_dtype == BITQ_DT_F32) {
        if (d.out_dtype == BITQ_DT_F32) launch_rope_layout<BITQ_DT_F32, BITQ_DT_F32>(a, pairs, vec, grid, st);
        else launch_rope_layout<BITQ_DT_F32, BITQ_DT_BF16>(a, pairs, vec, grid, st);
    } else {
        if (d.out_dtype == BITQ_DT_F32) launch_rope_layout<BITQ_DT_BF16, BITQ_DT_F32>(a, pairs, vec, grid, st);
        else launch_rope_layout<BITQ_DT_BF16, BITQ_DT_BF16>(a, pairs, vec, grid, st);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
