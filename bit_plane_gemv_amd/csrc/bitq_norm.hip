// Residual update of libbitq: the norm of a block's output, its gate and
// residual scale, and the next block's norm, in one pass.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitq_device.h"

namespace bitq {

// y = post u rsqrt(mean u^2 + e), r' = a r + b gate y, h = pre r' rsqrt(mean
// r'^2 + e): a row needs two sums over its elements, the second one of
// values that depend on the first.  W waves share a row and hold it in
// registers (NV chunks of 8 elements per lane), so u and r are read once and
// r' and h written once, whatever the number of passes the formulas take;
// all of a lane's loads, the weights' too, are issued before the first sum.
// Sums, r' and h are fp32; r' is rounded only where it is stored, and h is
// taken from the unrounded r'.  One wave per row needs no barrier (4 rows
// per workgroup); more waves meet in LDS.  Bound by HBM for many rows, by
// the latency of one round of loads and the reductions for few: 4096 rows of
// 8192 with a gate per token, bf16, 71 us (336 MB, 4.7 TB/s, the rate of a
// copy); with a gate per channel 56 us, with int8 rows out 59 (one more sum);
// one row of 4096, fp32, 3.7 us.
struct NormArgs {
    const void *u, *r, *post, *gate, *pre;
    void *ro, *h;
    float* d;
    int64_t us, rs, ros, hs, gs;
    float res, branch, eps_post, eps_pre;
    int M, C;
    int udt, rdt, wdt, odt;
    bool vec;  // every row chunk of 8 is 16-byte aligned
};

constexpr int kAnyType = -1;  // of rows that 16-byte loads cannot take: one kernel, types at run time

// 8 elements of a row as loaded (4 registers in bf16, 8 in fp32), converted
// where they are used: a row then stays in few enough registers for four or
// more rows per CU, and no load waits for another.  Elements k .. k + 7 of the
// row at `at`, the first n of them present (the rest 0).
//
// kAnyType: element e of the chunk is k + e T instead, so that the lanes of a
// load are neighbours (bf16, 1947 rows of 4231: 60 -> 25.5 us).
template <int DT>
struct Chunk {
    uint4 a[DT == BITQ_DT_F32 ? 2 : 1];
    __device__ __forceinline__ float at(int e, int) const {
        const uint4 q = a[DT == BITQ_DT_F32 ? e >> 2 : 0];
        const int w = DT == BITQ_DT_F32 ? e & 3 : e >> 1;
        const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
        if (DT == BITQ_DT_F32) return __uint_as_float(u);
        return __uint_as_float((e & 1) ? u & 0xFFFF0000u : u << 16);
    }
    __device__ __forceinline__ void load(const void* p, int, int64_t at, int k, int n, int, bool vec) {
        const int64_t i = at + k;
        if (DT == BITQ_DT_F32) {
            const float* f = static_cast<const float*>(p) + i;
            if (vec) {
                a[0] = reinterpret_cast<const uint4*>(f)[0];
                a[DT == BITQ_DT_F32 ? 1 : 0] = reinterpret_cast<const uint4*>(f)[1];
            } else {
                uint32_t u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = e < n ? __float_as_uint(f[e]) : 0u;
                a[0] = make_uint4(u[0], u[1], u[2], u[3]);
                a[DT == BITQ_DT_F32 ? 1 : 0] = make_uint4(u[4], u[5], u[6], u[7]);
            }
        } else {
            const uint16_t* f = static_cast<const uint16_t*>(p) + i;
            if (vec) {
                a[0] = *reinterpret_cast<const uint4*>(f);
            } else {
                uint32_t u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = e < n ? f[e] : 0u;
                a[0] = make_uint4(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
            }
        }
    }
    __device__ __forceinline__ void zero() {
        a[0] = make_uint4(0, 0, 0, 0);
        a[DT == BITQ_DT_F32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    }
};
// A row of C elements as a buffer of its bytes: elements past its end read as
// 0 and are not stored, so nothing has to be compared or masked.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* p, int64_t at, int C, int size) {
    return buffer_rsrc(static_cast<const uint8_t*>(p) + at * size, static_cast<uint32_t>(C * size));
}
template <>
struct Chunk<kAnyType> {
    uint32_t u[8];
    __device__ __forceinline__ float at(int e, int dt) const { return __uint_as_float(u[e] << (dt == BITQ_DT_F32 ? 0 : 16)); }
    __device__ __forceinline__ void load(const void* p, int dt, int64_t at, int k, int C, int step, bool) {
        if (dt == BITQ_DT_F32) {
            const auto b = row_buffer(p, at, C, 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = __builtin_amdgcn_raw_buffer_load_b32(b, 4 * (k + e * step), 0, 0);
        } else {
            const auto b = row_buffer(p, at, C, 2);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = __builtin_amdgcn_raw_buffer_load_b16(b, 2 * (k + e * step), 0, 0);
        }
    }
    __device__ __forceinline__ void zero() {}
};

__device__ __forceinline__ uint16_t norm_bf16(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ uint32_t norm_bf16x2(float a, float b) {
    return norm_bf16(a) | (static_cast<uint32_t>(norm_bf16(b)) << 16);
}

__device__ __forceinline__ void norm_store(void* p, int dt, int64_t i, int n, bool vec, const float (&v)[8]) {
    if (dt == BITQ_DT_F32) {
        float* f = static_cast<float*>(p) + i;
        if (vec) {
            reinterpret_cast<float4*>(f)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(f)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) f[e] = v[e];
        }
    } else if (dt == BITQ_DT_BF16) {
        uint16_t* f = static_cast<uint16_t*>(p) + i;
        if (vec) {
            *reinterpret_cast<uint4*>(f) = make_uint4(norm_bf16x2(v[0], v[1]), norm_bf16x2(v[2], v[3]),
                                                      norm_bf16x2(v[4], v[5]), norm_bf16x2(v[6], v[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) f[e] = norm_bf16(v[e]);
        }
    } else {  // int8 codes (integers held as floats)
        int8_t* f = static_cast<int8_t*>(p) + i;
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = static_cast<int>(v[e]);
        if (vec) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = (q[4 * j] & 255) | ((q[4 * j + 1] & 255) << 8) | ((q[4 * j + 2] & 255) << 16) |
                       (static_cast<uint32_t>(q[4 * j + 3]) << 24);
            *reinterpret_cast<uint2*>(f) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) f[e] = static_cast<int8_t>(q[e]);
        }
    }
}

__device__ __forceinline__ void norm_store_any(void* p, int dt, int64_t at, int k, int C, int step, const float (&v)[8]) {
    if (dt == BITQ_DT_F32) {
        const auto b = row_buffer(p, at, C, 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), b, 4 * (k + e * step), 0, 0);
    } else if (dt == BITQ_DT_BF16) {
        const auto b = row_buffer(p, at, C, 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) __builtin_amdgcn_raw_buffer_store_b16(norm_bf16(v[e]), b, 2 * (k + e * step), 0, 0);
    } else {
        const auto b = row_buffer(p, at, C, 1);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(static_cast<int>(v[e])), b, k + e * step, 0, 0);
    }
}

// The larger of two magnitudes, by their bits: NaN is the largest of all.
__device__ __forceinline__ float larger(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// Sum (or largest magnitude) over the W waves of a row, in a fixed order.
template <int W, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float t = __shfl_xor(v, o, 64);
        v = MAX ? larger(v, t) : v + t;
    }
    if constexpr (W > 1) {  // (s: a place that no wave can still be reading)
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if (lane == 0) s[wave] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = MAX ? larger(v, s[w]) : v + s[w];
    }
    return v;
}

template <int W, int NV, int UDT, int RDT, int WDT>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void block_norm_kernel(NormArgs a) {
    constexpr int T = 64 * W;                // lanes of a row
    constexpr bool ANY = UDT == kAnyType;    // lanes take neighbouring elements, T apart, instead of 8 in a row
    auto first = [&](int ln, int j) { return ANY ? 8 * T * j + ln : 8 * (ln + T * j); };
    // elements present of the chunk at i (<= 0: none); ANY: the row's buffer sees to that
    auto have = [&](int i) { return ANY ? a.C : min(8, a.C - i); };
    constexpr int RPB = W == 1 ? 4 : 1;      // rows of a workgroup
    // rows of 64 chunks and more per lane-group would not fit the registers
    // with r and the gate held from the start: these are then read late
    constexpr bool EARLY = NV * W < 64;
    // a place for each reduction of a row, for two rows in turn: a row has at
    // least one barrier, so no wave is more than a row behind
    __shared__ float s_red[2][3][W];
    const int ln = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int sub = W == 1 ? wave_uniform(threadIdx.x >> 6) : 0;
    int turn = 0;
    for (int next = blockIdx.x * RPB + sub; next < a.M; next += gridDim.x * RPB, turn ^= 1) {
        int row_ = wave_uniform(next);
        if constexpr (ANY) asm volatile("" : "+s"(row_));  // (one address of each buffer in the loop, not one for each element)
        const int64_t row = row_;
        Chunk<UDT> u[NV];
        Chunk<RDT> r[EARLY ? NV : 1];
        Chunk<WDT> g[EARLY ? NV : 1], po[1], pr[1];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = first(ln, j), n = have(i);
            const bool vec = !ANY && n == 8;
            u[j].zero();
            if (n <= 0) continue;
            u[j].load(a.u, a.udt, row * a.us, i, n, T, vec);
            if constexpr (EARLY) {
                if (a.r) r[j].load(a.r, a.rdt, row * a.rs, i, n, T, vec);
                if (a.gate) g[j].load(a.gate, a.wdt, row * a.gs, i, n, T, vec);
            }
            if constexpr (NV == 1) {
                if (a.post) po[0].load(a.post, a.wdt, 0, i, n, T, vec);
                if (a.pre) pr[0].load(a.pre, a.wdt, 0, i, n, T, vec);
            }
        }
        float s = a.branch;
        if (a.post) {
            float q = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) q = fmaf(u[j].at(e, a.udt), u[j].at(e, a.udt), q);
            q = row_reduce<W, false>(q, s_red[turn][0]);
            s *= 1.0f / sqrtf(q / static_cast<float>(a.C) + a.eps_post);
        }
        float y[NV][8], q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = first(ln, j), n = have(i);
            const bool vec = !ANY && n == 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[j][e] = u[j].at(e, a.udt) * s;
            if (n > 0) {
                constexpr int one = 0;
                if (a.post) {
                    if constexpr (NV > 1) po[0].load(a.post, a.wdt, 0, i, n, T, vec);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[j][e] *= po[0].at(e, a.wdt);
                }
                if (a.gate) {
                    const int k = EARLY ? j : one;
                    if constexpr (!EARLY) g[0].load(a.gate, a.wdt, row * a.gs, i, n, T, vec);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[j][e] *= g[k].at(e, a.wdt);
                }
                if (a.r) {
                    const int k = EARLY ? j : one;
                    if constexpr (!EARLY) r[0].load(a.r, a.rdt, row * a.rs, i, n, T, vec);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[j][e] = fmaf(a.res, r[k].at(e, a.rdt), y[j][e]);
                }
                if (a.ro) {
                    if constexpr (ANY) norm_store_any(a.ro, a.rdt, row * a.ros, i, n, T, y[j]);
                    else norm_store(a.ro, RDT, row * a.ros + i, n, vec, y[j]);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(y[j][e], y[j][e], q);
        }
        if (a.pre) {
            q = row_reduce<W, false>(q, s_red[turn][1]);
            const float f = 1.0f / sqrtf(q / static_cast<float>(a.C) + a.eps_pre);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = first(ln, j), n = have(i);
                if (n <= 0) continue;
                if constexpr (NV > 1) pr[0].load(a.pre, a.wdt, 0, i, n, T, !ANY && n == 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[j][e] = y[j][e] * f * pr[0].at(e, a.wdt);
            }
        }
        if (a.odt == BITQ_DT_ROW8) {  // the arithmetic of the activation quantizer
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) m = larger(m, fabsf(y[j][e]));
            m = row_reduce<W, true>(m, s_red[turn][2]);
            const float f = m > 0.0f ? __fdiv_rn(127.0f, m) : 0.0f;
            if (ln == 0) a.d[row] = __fdiv_rn(m, 127.0f);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[j][e] = __fmul_rn(y[j][e], f);
            if (!(m < INFINITY && f < INFINITY)) {
                // NaN: an infinity or NaN in the row, whose scale says so, or
                // a zero where 127 / m overflows (a branch, which other rows skip)
                asm volatile("");
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[j][e] = y[j][e] == y[j][e] ? y[j][e] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[j][e] = fminf(fmaxf(rintf(y[j][e]), -127.0f), 127.0f);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = first(ln, j), n = have(i);
            if constexpr (ANY) norm_store_any(a.h, a.odt, row * a.hs, i, n, T, y[j]);
            else if (n > 0) norm_store(a.h, a.odt, row * a.hs + i, n, n == 8, y[j]);
        }
    }
}

template <int W, int NV>
static void launch_norm(const NormArgs& a, hipStream_t st) {
    constexpr int rpb = W == 1 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.M + rpb - 1) / rpb, 1 << 16)));
    const dim3 block(W == 1 ? 256 : 64 * W);
    constexpr int F = BITQ_DT_F32, B = BITQ_DT_BF16, X = kAnyType;
    if (!a.vec) {
        hipLaunchKernelGGL((block_norm_kernel<W, NV, X, X, X>), grid, block, 0, st, a);
        return;
    }
    switch ((a.udt == B) * 4 + (a.rdt == B) * 2 + (a.wdt == B)) {
        case 0: hipLaunchKernelGGL((block_norm_kernel<W, NV, F, F, F>), grid, block, 0, st, a); break;
        case 1: hipLaunchKernelGGL((block_norm_kernel<W, NV, F, F, B>), grid, block, 0, st, a); break;
        case 2: hipLaunchKernelGGL((block_norm_kernel<W, NV, F, B, F>), grid, block, 0, st, a); break;
        case 3: hipLaunchKernelGGL((block_norm_kernel<W, NV, F, B, B>), grid, block, 0, st, a); break;
        case 4: hipLaunchKernelGGL((block_norm_kernel<W, NV, B, F, F>), grid, block, 0, st, a); break;
        case 5: hipLaunchKernelGGL((block_norm_kernel<W, NV, B, F, B>), grid, block, 0, st, a); break;
        case 6: hipLaunchKernelGGL((block_norm_kernel<W, NV, B, B, F>), grid, block, 0, st, a); break;
        default: hipLaunchKernelGGL((block_norm_kernel<W, NV, B, B, B>), grid, block, 0, st, a); break;
    }
}

int launch_block_norm(const bitq_norm_desc& d, const void* u, const void* r, const void* post, const void* gate,
                      const void* pre, void* ro, void* h, float* dscale, void* stream) {
    NormArgs a{u, r, post, gate, pre, ro, h, dscale, d.u_stride, d.r_stride, d.ro_stride, d.h_stride, d.gate_stride,
               d.res_scale, d.branch_scale, d.eps_post, d.eps_pre, d.rows, d.width, d.u_dtype, d.r_dtype, d.w_dtype,
               d.out_dtype, false};
    // chunks of 8 elements on their natural vector alignment in every row
    auto ok = [](const void* p, int dt, int64_t stride) {
        const int64_t e = dt == BITQ_DT_F32 ? 4 : dt == BITQ_DT_BF16 ? 2 : 1;
        const size_t al = dt == BITQ_DT_ROW8 ? 8 : 16;
        return !p || (aligned(p, al) && (stride * e) % static_cast<int64_t>(al) == 0);
    };
    a.vec = ok(u, d.u_dtype, d.u_stride) && ok(r, d.r_dtype, d.r_stride) && ok(ro, d.r_dtype, d.ro_stride) &&
            ok(post, d.w_dtype, 0) && ok(pre, d.w_dtype, 0) && ok(gate, d.w_dtype, d.gate_stride) &&
            ok(h, d.out_dtype, d.h_stride);
    const int chunks = (d.width + 7) / 8;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // few rows: one chunk a lane, for the shortest chain; many: fewer waves
    // with more of a row, for more rows at a time on a CU.  Measured, bf16, us:
    //   width 1024, <1,2> and <4,1>: 1024 rows 4.9 / 4.7, 2048 5.7 / 7.1
    //   2048, <1,4> (not kept) and <4,1>: 1024 rows 7.2 / 5.6, 4096 13.8 / 14.1
    //   4096, <4,2> and <16,1>: 256 rows 5.1 / 4.8, 512 6.0 / 8.0
    //   8192, <4,4> and <16,1>: 256 rows 7.6 / 6.0, 512 10.8 / 10.6, 1024 14.3 / 18.3
    const bool many = d.rows > 256;
    if (chunks <= 64) launch_norm<1, 1>(a, st);
    else if (d.rows > 1024 && chunks <= 128) launch_norm<1, 2>(a, st);
    else if (chunks <= 256) launch_norm<4, 1>(a, st);
    else if (many && chunks <= 512) launch_norm<4, 2>(a, st);
    else if (many && chunks <= 1024) launch_norm<4, 4>(a, st);
    else if (chunks <= 1024) launch_norm<16, 1>(a, st);
    else if (chunks <= 2048) launch_norm<16, 2>(a, st);
    else launch_norm<16, 4>(a, st);
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
