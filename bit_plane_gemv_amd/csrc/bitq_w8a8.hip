// Int8 matrix product of libbitq with a scale per token and output channel.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitq_device.h"

namespace bitq {

// y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k]: both operands have k
// contiguous, which is how the int8 matrix instructions take them (a lane's
// 16 bytes are 16 consecutive k of one row).  Sums are int32 and exact
// (K <= 131056), so no order of summation matters; the scales are applied to
// the converted sum in fp32.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

struct GemmArgs {
    const int8_t* a;
    const int8_t* w;
    const float *sa, *sw;
    void* y;
    int64_t lda, ldw, ldy;
    int M, N, K;
    int out;  // 0 fp32, 1 bf16, 2 int32 sums
};

__device__ __forceinline__ void put(const GemmArgs& g, int64_t m, int n, int acc, float sa, float sw) {
    const int64_t i = m * g.ldy + n;
    if (g.out == 2) {
        static_cast<int32_t*>(g.y)[i] = acc;
    } else {
        const float v = static_cast<float>(acc) * sa * sw;
        if (g.out == 0) static_cast<float*>(g.y)[i] = v;
        else static_cast<uint16_t*>(g.y)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
}

constexpr uint32_t kOutOfRange = 0x80000000u;  // offset past every descriptor's range: the load returns zeros

// ------------------------------------------------------------ few tokens
// At most 64 tokens: bound by the weight stream.  A workgroup owns 16 output
// channels over the whole k range; its KW waves take 128-byte pieces of k
// round-robin, U of them loaded together, straight from memory into the
// operands of v_mfma_i32_16x16x64_i8 (A = 16 weight rows, B = 16 tokens, TT
// token tiles), and add their sums in LDS.
template <int TT, int KW, int U>
__global__ __launch_bounds__(64 * KW) void w8a8_few_kernel(GemmArgs g) {
    __shared__ int s_part[KW][TT][4][68];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int grp = lane >> 4, j = lane & 15;
    const int n0 = 16 * blockIdx.x;
    const int rows = min(16, g.N - n0);
    const auto rw = buffer_rsrc(g.w + n0 * g.ldw, static_cast<uint32_t>((rows - 1) * g.ldw + g.K));
    const auto ra = buffer_rsrc(g.a, static_cast<uint32_t>((g.M - 1) * g.lda + g.K));
    const uint32_t wo = j < rows ? static_cast<uint32_t>(j * g.ldw) + 16 * grp : kOutOfRange;
    uint32_t ao[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) ao[t] = 16 * t + j < g.M ? static_cast<uint32_t>((16 * t + j) * g.lda) + 16 * grp : kOutOfRange;
    i32x4_t acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = i32x4_t{0, 0, 0, 0};
    auto vec = [](uint4 u) {
        return i32x4_t{static_cast<int>(u.x), static_cast<int>(u.y), static_cast<int>(u.z), static_cast<int>(u.w)};
    };
    for (int k0 = 128 * wave; k0 < g.K; k0 += 128 * KW * U) {
        i32x4_t wv[U][2], av[U][2][TT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = k0 + 128 * KW * u + 64 * s;
                const bool in = k + 16 * grp < g.K;  // (K is a multiple of 16)
                wv[u][s] = vec(buffer_load_u128(rw, in ? wo + k : kOutOfRange, 0));
#pragma unroll
                for (int t = 0; t < TT; ++t) av[u][s][t] = vec(buffer_load_u128(ra, in ? ao[t] + k : kOutOfRange, 0));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][s], av[u][s][t], acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_part[wave][t][i][lane] = acc[t][i];
    __syncthreads();
    // output (channel n0 + 4 gq + i, token 16 t + j) is element i of lane 16 gq + j
    for (int idx = tid; idx < TT * 256; idx += 64 * KW) {
        const int c = idx & 15, jj = (idx >> 4) & 15, t = idx >> 8;
        const int n = n0 + c, m = 16 * t + jj;
        int v = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w) v += s_part[w][t][c & 3][16 * (c >> 2) + jj];
        if (n < g.N && m < g.M) put(g, m, n, v, g.out == 2 ? 0.0f : g.sa[m], g.out == 2 ? 0.0f : g.sw[n]);
    }
}

// ----------------------------------------------------------- many tokens
// Tiles of BM tokens x BN channels, k in stages of 128 bytes copied straight
// from memory into LDS (two stages, the next one in flight while one is
// multiplied).  A row of a stage is 128 bytes in LDS; its 16-byte pieces are
// stored at position p ^ (row & 7), so that the operand reads of 16 or 32
// consecutive rows spread over the banks.  The copy writes LDS in lane
// order, so the permutation is applied to the addresses it reads.
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void w8a8_tile_kernel(GemmArgs g, int tiles_m, int tiles_n) {
    constexpr int WAVES = (BM / WM) * (BN / WN), BK = 128;
    constexpr int TM = WM / 32, TN = WN / 32;
    constexpr int ROWS = BM + BN, PER = ROWS / 8 / WAVES;  // 8-row copies per wave and stage
    static_assert(ROWS % (8 * WAVES) == 0 && BM % 8 == 0, "copies divide evenly");
    __shared__ __align__(1024) uint8_t s_t[2][ROWS * BK];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    // tile of this workgroup: each XCD (blockIdx % 8) takes a contiguous
    // range of tiles, in columns of 8 token tiles
    const int total = tiles_m * tiles_n, per = total / 8, extra = total % 8, xcd = blockIdx.x % 8;
    const int id = xcd * per + min(xcd, extra) + blockIdx.x / 8;
    const int gcol = id / (8 * tiles_n), gm = min(8, tiles_m - 8 * gcol), rem = id - gcol * 8 * tiles_n;
    const int m0 = (8 * gcol + rem % gm) * BM, n0 = (rem / gm) * BN;
    const int rm = min(BM, g.M - m0), rn = min(BN, g.N - n0);
    const auto ra = buffer_rsrc(g.a + m0 * g.lda, static_cast<uint32_t>((rm - 1) * g.lda + g.K));
    const auto rw = buffer_rsrc(g.w + n0 * g.ldw, static_cast<uint32_t>((rn - 1) * g.ldw + g.K));
    // this wave's copies: rows 8 (wave PER + i) .. + 7 of the stage (tokens first)
    const int piece = (lane & 7) ^ (lane >> 3);  // k piece this lane reads (row & 7 = lane / 8)
    uint32_t off[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int row = 8 * (wave * PER + i) + (lane >> 3);
        if (8 * (wave * PER + i) < BM) off[i] = row < rm ? static_cast<uint32_t>(row * g.lda) + 16 * piece : kOutOfRange;
        else off[i] = row - BM < rn ? static_cast<uint32_t>((row - BM) * g.ldw) + 16 * piece : kOutOfRange;
    }
    auto copy = [&](int k0, int buf) __attribute__((always_inline)) {
        const bool in = k0 + 16 * piece < g.K;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool isa = 8 * (wave * PER + i) < BM;
            buffer_copy_lds16(isa ? ra : rw, &s_t[buf][(wave * PER + i) * 1024], in ? off[i] + k0 : kOutOfRange);
        }
    };
    i32x16_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int jn = 0; jn < TN; ++jn)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][jn][e] = 0;
    const int half = lane >> 5, r32 = lane & 31;
    copy(0, 0);
    int buf = 0;
    for (int k0 = 0; k0 < g.K; k0 += BK) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (k0 + BK < g.K) copy(k0 + BK, buf ^ 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            i32x4_t av[TM], wv[TN];
            const int pc = 2 * ks + half;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = wm * WM + 32 * i + r32;
                av[i] = *reinterpret_cast<const i32x4_t*>(&s_t[buf][row * BK + ((pc ^ (row & 7)) << 4)]);
            }
#pragma unroll
            for (int jn = 0; jn < TN; ++jn) {
                const int row = BM + wn * WN + 32 * jn + r32;
                wv[jn] = *reinterpret_cast<const i32x4_t*>(&s_t[buf][row * BK + ((pc ^ (row & 7)) << 4)]);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int jn = 0; jn < TN; ++jn)
                    acc[i][jn] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[i], wv[jn], acc[i][jn], 0, 0, 0);
        }
        buf ^= 1;
    }
    // element e of lane l: token 8 (e / 4) + 4 (l / 32) + e % 4, channel l % 32
#pragma unroll
    for (int jn = 0; jn < TN; ++jn) {
        const int n = n0 + wn * WN + 32 * jn + r32;
        const float sw = g.out != 2 && n < g.N ? g.sw[n] : 0.0f;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int m = m0 + wm * WM + 32 * i + 8 * (e >> 2) + 4 * half + (e & 3);
                if (m < g.M && n < g.N) put(g, m, n, acc[i][jn][e], g.out != 2 ? g.sa[m] : 0.0f, sw);
            }
    }
}

W8A8Plan w8a8_plan(const bitq_w8a8_desc& d) {
    W8A8Plan p{};
    p.kernel = d.M <= 64 ? (d.M + 15) / 16 : 5;
    p.splits = 1;
    p.ws_bytes = 0;
    return p;
}

template <int BM, int BN, int WM, int WN>
static void launch_tile(const GemmArgs& g, hipStream_t st) {
    const int tm = (g.M + BM - 1) / BM, tn = (g.N + BN - 1) / BN;
    hipLaunchKernelGGL((w8a8_tile_kernel<BM, BN, WM, WN>), dim3(static_cast<unsigned>(tm) * tn),
                       dim3(64 * (BM / WM) * (BN / WN)), 0, st, g, tm, tn);
}

int launch_gemm_w8a8(const bitq_w8a8_desc& d, const W8A8Plan& plan, const void* a, const float* sa, const void* w,
                     const float* sw, void* y, void* ws, void* stream) {
    const GemmArgs g{static_cast<const int8_t*>(a), static_cast<const int8_t*>(w), sa, sw, y, d.lda, d.ldw, d.ldy,
                     d.M, d.N, d.K, (d.flags & BITQ_F_ACC_INT32) ? 2 : d.y_dtype == BITQ_DT_BF16 ? 1 : 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 few(static_cast<unsigned>((d.N + 15) / 16));
    switch (plan.kernel) {
        case 1: hipLaunchKernelGGL((w8a8_few_kernel<1, 8, 4>), few, dim3(512), 0, st, g); break;
        case 2: hipLaunchKernelGGL((w8a8_few_kernel<2, 8, 4>), few, dim3(512), 0, st, g); break;
        case 3: hipLaunchKernelGGL((w8a8_few_kernel<3, 8, 2>), few, dim3(512), 0, st, g); break;
        case 4: hipLaunchKernelGGL((w8a8_few_kernel<4, 8, 2>), few, dim3(512), 0, st, g); break;
        default: launch_tile<128, 128, 64, 64>(g, st); break;
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
