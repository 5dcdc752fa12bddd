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
// the latency of one round of loads and the reductions for few.
struct NormArgs {
    const void *u, *r, *post, *gate, *pre;
    void *ro, *h;
    float* d;
    int64_t us, rs, ros, hs, gs;
    float res, branch, eps_post, eps_pre;
    int M, C;
    int udt, rdt, wdt, odt;
    bool vec;  // every row chunk of 8 is 16-byte aligned, and C a multiple of 8
};

__device__ __forceinline__ void norm_load(const void* p, int dt, int64_t i, int n, bool vec, float (&v)[8]) {
    if (dt == BITQ_DT_F32) {
        const float* f = static_cast<const float*>(p) + i;
        if (vec) {
            const float4 a = reinterpret_cast<const float4*>(f)[0], b = reinterpret_cast<const float4*>(f)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? f[e] : 0.0f;
        }
    } else {
        const uint16_t* f = static_cast<const uint16_t*>(p) + i;
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4*>(f);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(w[e] << 16);
                v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? bf16_to_f32(f[e]) : 0.0f;
        }
    }
}

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

// Sum (or maximum) over the W waves of a row, in a fixed order.
template <int W, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float t = __shfl_xor(v, o, 64);
        v = MAX ? fmaxf(v, t) : v + t;
    }
    if constexpr (W > 1) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        __syncthreads();  // (reads of the previous reduction are done)
        if (lane == 0) s[wave] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = MAX ? fmaxf(v, s[w]) : v + s[w];
    }
    return v;
}

template <int W, int NV>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void block_norm_kernel(NormArgs a) {
    constexpr int T = 64 * W;                // lanes of a row
    constexpr int RPB = W == 1 ? 4 : 1;      // rows of a workgroup
    __shared__ float s_red[W];
    const int ln = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int sub = W == 1 ? threadIdx.x >> 6 : 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + sub; row < a.M; row += static_cast<int64_t>(gridDim.x) * RPB) {
        float u[NV][8], r[NV][8], g[NV][8], po[NV][8], pr[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = 8 * (ln + T * j), n = min(8, a.C - i);  // elements of this chunk (<= 0: none)
            const bool vec = a.vec && n == 8;
            if (n > 0) {
                norm_load(a.u, a.udt, row * a.us + i, n, vec, u[j]);
                if (a.r) norm_load(a.r, a.rdt, row * a.rs + i, n, vec, r[j]);
                if (a.gate) norm_load(a.gate, a.wdt, row * a.gs + i, n, vec, g[j]);
                if (a.post) norm_load(a.post, a.wdt, i, n, vec, po[j]);
                if (a.pre) norm_load(a.pre, a.wdt, i, n, vec, pr[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] = r[j][e] = g[j][e] = po[j][e] = pr[j][e] = 0.0f;
            }
        }
        if (a.post) {
            float q = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) q = fmaf(u[j][e], u[j][e], q);
            q = row_reduce<W, false>(q, s_red);
            const float s = 1.0f / sqrtf(q / static_cast<float>(a.C) + a.eps_post);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] = u[j][e] * s * po[j][e];
        }
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = a.branch * u[j][e];
                if (a.gate) y *= g[j][e];
                if (a.r) y = fmaf(a.res, r[j][e], y);
                u[j][e] = y;
                q = fmaf(y, y, q);
            }
        if (a.ro) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = 8 * (ln + T * j), n = min(8, a.C - i);
                if (n > 0) norm_store(a.ro, a.rdt, row * a.ros + i, n, a.vec && n == 8, u[j]);
            }
        }
        if (a.pre) {
            q = row_reduce<W, false>(q, s_red);
            const float s = 1.0f / sqrtf(q / static_cast<float>(a.C) + a.eps_pre);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] = u[j][e] * s * pr[j][e];
        }
        if (a.odt == BITQ_DT_ROW8) {  // the arithmetic of the activation quantizer
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(u[j][e]));
            m = row_reduce<W, true>(m, s_red);
            const float s = m > 0.0f ? __fdiv_rn(127.0f, m) : 0.0f;
            if (ln == 0) a.d[row] = m > 0.0f ? __fdiv_rn(m, 127.0f) : 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[j][e] = fminf(fmaxf(rintf(__fmul_rn(u[j][e], s)), -127.0f), 127.0f);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = 8 * (ln + T * j), n = min(8, a.C - i);
            if (n > 0) norm_store(a.h, a.odt, row * a.hs + i, n, a.vec && n == 8, u[j]);
        }
    }
}

template <int W>
static void launch_norm(const NormArgs& a, int nv, hipStream_t st) {
    constexpr int rpb = W == 1 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.M + rpb - 1) / rpb, 1 << 16)));
    const dim3 block(W == 1 ? 256 : 64 * W);
    if (nv <= 1) hipLaunchKernelGGL((block_norm_kernel<W, 1>), grid, block, 0, st, a);
    else if (nv <= 2) hipLaunchKernelGGL((block_norm_kernel<W, 2>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((block_norm_kernel<W, 4>), grid, block, 0, st, a);
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
    // many rows: the fewest waves that hold a row with 4 chunks a lane; few
    // rows: one chunk a lane, for the shortest chain
    const int per = d.rows >= 1024 ? 4 : 1;
    int W = 1;
    while (W < 16 && 64 * W * per < chunks) W *= 2;
    const int nv = (chunks + 64 * W - 1) / (64 * W);
    hipStream_t st = static_cast<hipStream_t>(stream);
    switch (W) {
        case 1: launch_norm<1>(a, nv, st); break;
        case 2: launch_norm<2>(a, nv, st); break;
        case 4: launch_norm<4>(a, nv, st); break;
        case 8: launch_norm<8>(a, nv, st); break;
        default: launch_norm<16>(a, nv, st); break;
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
