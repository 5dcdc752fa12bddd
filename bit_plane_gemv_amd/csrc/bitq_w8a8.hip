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
//
// Both kernels feed v_mfma_i32_16x16x64_i8 (A = 16 weight rows, B = 16
// tokens: a lane then holds 4 consecutive channels of one token) from LDS,
// which is filled by copies straight from memory.  A row of a stage is
// ROWB = 64 or 128 bytes of k there, so one copy instruction (lane l writes
// bytes 16 l .. 16 l + 15) brings 16 or 8 rows, and lane 16 g + r of an
// operand read takes a 16-byte piece of row r.  Piece p of row r is stored at
// place p ^ (-(r / 4) mod 4) of the row's four, or p ^ (r mod 8) of its eight,
// which keeps the operand reads free of bank conflicts (counted: none); the
// copy applies the permutation to the addresses it reads.
typedef int i32x4_t __attribute__((ext_vector_type(4)));

struct GemmArgs {
    const int8_t* a;
    const int8_t* w;
    const float *sa, *sw;
    void* y;
    int64_t lda, ldw, ldy;
    int M, N, K;
    int out;  // 0 fp32, 1 bf16, 2 int32 sums
};

constexpr uint32_t kOutOfRange = 0x80000000u;  // offset past every descriptor's range: the load returns zeros

// Byte of row r at which its 16-byte piece p is stored (also its own inverse
// in p, as the copies use it).
template <int ROWB>
__device__ __forceinline__ uint32_t place(int r, int p) {
    return static_cast<uint32_t>(ROWB == 64 ? p ^ (-(r >> 2) & 3) : p ^ (r & 7)) << 4;
}

// At most N of this wave's memory operations still outstanding.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}

// y of one output (few-token kernel)
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

// ------------------------------------------------------------ few tokens
// At most 64 tokens: bound by the weight stream (one token, 11008 x 4096: 9.5
// us, 4.7 TB/s; 28672 x 8192: 40.7 us, 5.8 TB/s).  A workgroup owns NB tiles
// of 16 channels over the whole k range; its KW waves take units of k
// round-robin, and add their sums in LDS at the end.  A wave has a ring of NS
// units of its own in LDS, so the waves never wait for each other: the wave
// keeps NS - 1 units of copies in flight and waits for the oldest one only.
//
// TC = 1: at most 8 tokens, one copy brings them (rows 8 .. 15 of the tile
// then hold another unit's bytes; their products are not stored).
template <int TT, int NB, int KW, int NS, int TC = 2 * TT>
__global__ __launch_bounds__(64 * KW) void w8a8_few_kernel(GemmArgs g) {
    static_assert(TC == 2 * TT || (TT == 1 && TC == 1), "two copies a tile, or one of 8 tokens");
    constexpr int ROWB = 128, PER = 2 * NB + TC, UNIT = PER * 1024;  // copies and bytes of a unit (2 copies a tile)
    constexpr int SUMS = KW * TT * NB * 4 * 68 * 4;
    constexpr int RINGS = KW * NS * UNIT + (TC == 1 ? 1024 : 0);  // (TC = 1: the last unit's missing rows lie past it)
    __shared__ __align__(1024) uint8_t s_mem[RINGS > SUMS ? RINGS : SUMS];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int grp = lane >> 4, r = lane & 15;
    const int n0 = 16 * NB * blockIdx.x;
    const int rows = min(16 * NB, g.N - n0);
    const auto rw = buffer_rsrc(g.w + n0 * g.ldw, static_cast<uint32_t>((rows - 1) * g.ldw + g.K));
    const auto ra = buffer_rsrc(g.a, static_cast<uint32_t>((g.M - 1) * g.lda + g.K));
    const int crow = lane >> 3, piece = static_cast<int>(place<ROWB>(crow, lane & 7) >> 4);
    uint32_t off[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int row = 8 * i + crow;
        if (i < 2 * NB) off[i] = row < rows ? static_cast<uint32_t>(row * g.ldw) + 16 * piece : kOutOfRange;
        else off[i] = row - 16 * NB < g.M ? static_cast<uint32_t>((row - 16 * NB) * g.lda) + 16 * piece : kOutOfRange;
    }
    uint8_t* ring = s_mem + wave * (NS * UNIT);
    auto copy = [&](int k, int slot) __attribute__((always_inline)) {
        const bool in = k + 16 * piece < g.K;  // (K is a multiple of 16)
#pragma unroll
        for (int i = 0; i < PER; ++i) buffer_copy_lds16(i < 2 * NB ? rw : ra, ring + slot * UNIT + i * 1024, in ? off[i] + k : kOutOfRange);
    };
    i32x4_t acc[NB][TT];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[i][t] = i32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) copy(ROWB * (wave + KW * s), s);
    const uint32_t at[2] = {r * ROWB + place<ROWB>(r, grp), r * ROWB + place<ROWB>(r, 4 + grp)};
    int slot = 0, next = NS - 1;
    for (int k = ROWB * wave; k < g.K; k += ROWB * KW) {
        wait_copies<(NS - 2) * PER>();
        i32x4_t wv[2][NB], av[2][TT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < NB; ++i) wv[s][i] = *reinterpret_cast<const i32x4_t*>(ring + slot * UNIT + i * 2048 + at[s]);
#pragma unroll
            for (int t = 0; t < TT; ++t) av[s][t] = *reinterpret_cast<const i32x4_t*>(ring + slot * UNIT + (NB + t) * 2048 + at[s]);
        }
        // (into the slot read in the previous turn: its reads were waited for by its products)
        copy(k + ROWB * KW * (NS - 1), next);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[s][i], av[s][t], acc[i][t], 0, 0, 0);
        slot = slot + 1 == NS ? 0 : slot + 1;
        next = next + 1 == NS ? 0 : next + 1;
    }
    // ---- the waves' sums (the copies past K still write the rings)
    wait_copies<0>();
    __syncthreads();
    int (*s_part)[NB * TT * 4][68] = reinterpret_cast<int (*)[NB * TT * 4][68]>(s_mem);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s_part[wave][(i * TT + t) * 4 + e][lane] = acc[i][t][e];
    __syncthreads();
    // output (channel n0 + 16 i + 4 q + e, token 16 t + j) is element e of lane 16 q + j
    for (int idx = tid; idx < NB * TT * 256; idx += 64 * KW) {
        const int c = idx & 15, j = (idx >> 4) & 15, it = idx >> 8;
        const int n = n0 + 16 * (it / TT) + c, m = 16 * (it % TT) + j;
        if (n >= g.N || m >= g.M) continue;
        int v = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w) v += s_part[w][it * 4 + (c & 3)][16 * (c >> 2) + j];
        put(g, m, n, v, g.out == 2 ? 0.0f : g.sa[m], g.out == 2 ? 0.0f : g.sw[n]);
    }
}

// ----------------------------------------------------------- many tokens
// Tiles of BM tokens x BN channels in a ring of NS stages of KSUB units of k;
// wave tiles of WM x WN.  The copies run NS - 1 stages ahead, the operand
// reads one unit ahead of the products (a second set of operand registers),
// and the workgroup meets once per stage.  Many tokens: bound by the matrix
// cores and LDS, which a 256 x 256 tile loads alike (1024 cycles of products,
// 768 of operand reads and 256 of copies per unit), at the clock that their
// power allows: 4096 x 8192 x 8192 231 us, 2.38 POP/s, what a library product
// of 8192^3 reaches; 4096 x 11008 x 4096 170 us in a run of 1500 calls, 177 a
// call with pauses of 10 ms, 190 - 200 in the first 20 calls after a pause (a
// library's product without scales: 179, 203 and 203 - 209 there), its
// 688 tiles filling 2.7 of 3 rounds.  (Waves of 128 x 128, with fewer operand
// reads, but one to a SIMD: 198 us.)  Few tokens: bound by the weight stream
// and the ramp of its few workgroups (64 x 4096 x 11008: 10 us and the join's 4).
//
// The tile's outputs go through LDS, a wave's part of it at a time, and leave
// as 16-byte stores of whole 128-byte lines.
template <int ES, int WM, int WN>
__device__ __forceinline__ void store_tile(const GemmArgs& g, i32x4_t (&acc)[WM / 16][WN / 16], uint8_t* mem, int mw, int nw,
                                           int lane) {
    constexpr int TM = WM / 16, TN = WN / 16;
    constexpr int STEP = TM < (ES == 2 ? 4 : 2) ? TM : (ES == 2 ? 4 : 2);  // 16-token tiles at a time
    constexpr int RS = WN * ES + 16;                                       // bytes of a row in LDS
    constexpr int LPR = WN * ES / 16, RPI = 64 / LPR;                      // lanes of a row, rows of a store
    const int grp = lane >> 4, r = lane & 15;
    uint8_t* y = static_cast<uint8_t*>(g.y);
    const bool vec = (reinterpret_cast<uintptr_t>(y) & 15) == 0 && (g.ldy * ES) % 16 == 0 && nw + WN <= g.N;
    float sw[TN][4];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sw[j][e] = g.out == 2 ? 0.0f : g.sw[min(nw + 16 * j + 4 * grp + e, g.N - 1)];
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += STEP) {
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
            const float sa = g.out == 2 ? 0.0f : g.sa[min(mw + 16 * (i0 + i) + r, g.M - 1)];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                uint8_t* p = mem + (16 * i + r) * RS + (16 * j + 4 * grp) * ES;
                const i32x4_t c = acc[i0 + i][j];
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(c[e]) * sa * sw[j][e];
                if constexpr (ES == 2) {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e]));
                    *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
                } else if (g.out == 2) {
                    *reinterpret_cast<i32x4_t*>(p) = c;
                } else {
                    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        wait_lds();  // (the part of LDS is this wave's own)
        if (vec) {
#pragma unroll
            for (int q = 0; q < 16 * STEP / RPI; ++q) {
                const int row = q * RPI + lane / LPR, m = mw + 16 * i0 + row;
                const uint4 u = *reinterpret_cast<const uint4*>(mem + row * RS + (lane % LPR) * 16);
                if (m < g.M) *reinterpret_cast<uint4*>(y + (m * g.ldy + nw) * ES + (lane % LPR) * 16) = u;
            }
        } else {
            for (int q = lane; q < 16 * STEP * WN; q += 64) {
                const int row = q / WN, c = q % WN, m = mw + 16 * i0 + row, n = nw + c;
                if (m < g.M && n < g.N) {
                    if constexpr (ES == 2)
                        reinterpret_cast<uint16_t*>(y)[m * g.ldy + n] = *reinterpret_cast<const uint16_t*>(mem + row * RS + c * 2);
                    else
                        reinterpret_cast<uint32_t*>(y)[m * g.ldy + n] = *reinterpret_cast<const uint32_t*>(mem + row * RS + c * 4);
                }
            }
        }
        wait_lds();
    }
}

template <int BM, int BN, int WM, int WN, int NS, int KSUB>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) void w8a8_tile_kernel(GemmArgs g, int tiles_m, int tiles_n,
                                                                                int splits, int kper, int* ws) {
    constexpr int WAVES = (BM / WM) * (BN / WN), TM = WM / 16, TN = WN / 16;
    constexpr int ROWB = 64 * KSUB, ROWS = BM + BN, STAGE = ROWS * ROWB;
    constexpr int CR = 1024 / ROWB, PER = ROWS / CR / WAVES;  // rows of a copy, copies per wave of a stage
    static_assert(KSUB == 1 || KSUB == 2, "rows of 64 or 128 bytes");
    static_assert(BM % (CR * WAVES) == 0 && BN % (CR * WAVES) == 0, "a copy slot is all tokens or all channels");
    static_assert(NS >= 3, "a stage is copied while one is read and one is waited for");
    constexpr int PART2 = 16 * (TM < 4 ? TM : 4) * (WN * 2 + 16), PART4 = 16 * (TM < 2 ? TM : 2) * (WN * 4 + 16);
    constexpr int PART = PART2 > PART4 ? PART2 : PART4;  // a wave's part of LDS for its outputs
    static_assert(WAVES * PART <= NS * STAGE, "the outputs pass through the ring");
    extern __shared__ __align__(1024) uint8_t s_ring[];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    // tile of this workgroup: each XCD (blockIdx % 8) takes a contiguous
    // range of tiles, in columns of 4 token tiles, so that the tiles it works
    // on at a time share their rows in its L2
    const int total = tiles_m * tiles_n, bid = static_cast<int>(blockIdx.x) / splits, part_k = static_cast<int>(blockIdx.x) % splits;
    const int per = total / 8, extra = total % 8, xcd = bid % 8;
    const int id = xcd * per + min(xcd, extra) + bid / 8;
    const int col = id / (4 * tiles_n), cm = min(4, tiles_m - 4 * col), rem = id - col * 4 * tiles_n;
    const int m0 = (4 * col + rem % cm) * BM, n0 = (rem / cm) * BN;
    const int rm = min(BM, g.M - m0), rn = min(BN, g.N - n0);
    const auto ra = buffer_rsrc(g.a + m0 * g.lda, static_cast<uint32_t>((rm - 1) * g.lda + g.K));
    const auto rw = buffer_rsrc(g.w + n0 * g.ldw, static_cast<uint32_t>((rn - 1) * g.ldw + g.K));
    const int kbeg = part_k * kper, kend = min(g.K, kbeg + kper);  // (kper: a multiple of 128)
    const int crow = lane / (64 / CR), piece = static_cast<int>(place<ROWB>(crow, lane % (64 / CR)) >> 4);
    uint32_t off[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int row = CR * (wave + WAVES * i) + crow;
        if (CR * WAVES * i < BM) off[i] = row < rm ? static_cast<uint32_t>(row * g.lda) + 16 * piece : kOutOfRange;
        else off[i] = row - BM < rn ? static_cast<uint32_t>((row - BM) * g.ldw) + 16 * piece : kOutOfRange;
    }
    auto copy = [&](int k, int stage) __attribute__((always_inline)) {
        const bool in = k + 16 * piece < kend;  // (K is a multiple of 16)
#pragma unroll
        for (int i = 0; i < PER; ++i)
            buffer_copy_lds16(CR * WAVES * i < BM ? ra : rw, s_ring + stage * STAGE + (wave + WAVES * i) * 1024,
                              in ? off[i] + k : kOutOfRange);
    };
    i32x4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
    const int grp = lane >> 4, r = lane & 15;
    const uint32_t arow = (wm * WM + r) * ROWB, wrow = (BM + wn * WN + r) * ROWB;
    i32x4_t av[2][TM], wv[2][TN];
    auto operands = [&](int stage, int u, int f) __attribute__((always_inline)) {
        const uint8_t* b = s_ring + stage * STAGE + place<ROWB>(r, 4 * u + grp);
#pragma unroll
        for (int j = 0; j < TN; ++j) wv[f][j] = *reinterpret_cast<const i32x4_t*>(b + wrow + 16 * ROWB * j);
#pragma unroll
        for (int i = 0; i < TM; ++i) av[f][i] = *reinterpret_cast<const i32x4_t*>(b + arow + 16 * ROWB * i);
    };
    auto products = [&](int f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[f][j], av[f][i], acc[i][j], 0, 0, 0);
    };
    int cur = 0, nxt = 1, cpy = NS - 1;  // stages: multiplied, read next, copied into
    // One unit: the next unit's operands are read (and, at a stage's end, the
    // stage after the ring's last is copied) while this one is multiplied.
    // The stage copied into was read before the last meeting.
    auto unit = [&](int k0, int u, int f) __attribute__((always_inline)) {
        const bool last = u == KSUB - 1;
        if (last) {
            wait_copies<(NS - 3) * PER>();  // this wave's copies of stage nxt have landed
            __builtin_amdgcn_s_barrier();   // and everyone's
            asm volatile("" ::: "memory");
            operands(nxt, 0, f ^ 1);
            copy(k0 + ROWB * (NS - 1), cpy);
        } else {
            operands(cur, u + 1, f ^ 1);
        }
        products(f);
        if constexpr (TM * TN >= 32 && KSUB == 1) {
            // operand reads and copies spread among the products (256 x 256
            // tiles: 8 % fewer cycles than in the compiler's order)
#pragma unroll
            for (int i = 0; i < TM + TN; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            }
        }
        if (last) {
            cur = nxt;
            nxt = nxt + 1 == NS ? 0 : nxt + 1;
            cpy = cpy + 1 == NS ? 0 : cpy + 1;
        }
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) copy(kbeg + ROWB * s, s);
    wait_copies<(NS - 2) * PER>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    operands(0, 0, 0);
    for (int k0 = kbeg; k0 < kend; k0 += 128) {  // (two units a turn: the operand registers alternate; past the end they hold zeros)
#pragma unroll
        for (int v = 0; v < 2; ++v) unit(k0 + ROWB * (v / KSUB), v % KSUB, v & 1);
    }
    wait_copies<0>();  // no copy lands in the outputs' place
    __syncthreads();
    if (splits > 1) {  // this k range's sums, in the order in which the lanes hold them, for w8a8_join_kernel
        int* mine = ws + ((static_cast<int64_t>(part_k) * total + id) * WAVES + wave) * (TM * TN * 256) + lane * 4;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) *reinterpret_cast<i32x4_t*>(mine + (i * TN + j) * 256) = acc[i][j];
        return;
    }
    uint8_t* part = s_ring + wave * PART;
    if (g.out == 1) store_tile<2, WM, WN>(g, acc, part, m0 + wm * WM, n0 + wn * WN, lane);
    else store_tile<4, WM, WN>(g, acc, part, m0 + wm * WM, n0 + wn * WN, lane);
}

// Adds the sums of a tile's k ranges (int32: exact in any order) and writes
// y: one lane per 4 channels of a token, as the tile kernel's lanes hold them.
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256) void w8a8_join_kernel(GemmArgs g, int tiles_m, int tiles_n, int splits, const int* __restrict__ ws) {
    constexpr int WAVES = (BM / WM) * (BN / WN), TN = WN / 16, PER_TILE = BM * BN / 4;
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // (a tile is whole workgroups)
    const int total = tiles_m * tiles_n, id = static_cast<int>(q / PER_TILE), in = static_cast<int>(q % PER_TILE);
    i32x4_t v = {0, 0, 0, 0};
    const int64_t step = static_cast<int64_t>(total) * PER_TILE;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) v += reinterpret_cast<const i32x4_t*>(ws)[s * step + q];
    const int lane = in & 63, ij = (in >> 6) % (PER_TILE / 64 / WAVES), wave = (in >> 6) / (PER_TILE / 64 / WAVES);
    const int col = id / (4 * tiles_n), cm = min(4, tiles_m - 4 * col), rem = id - col * 4 * tiles_n;
    const int m = (4 * col + rem % cm) * BM + (wave % (BM / WM)) * WM + 16 * (ij / TN) + (lane & 15);
    const int n = (rem / cm) * BN + (wave / (BM / WM)) * WN + 16 * (ij % TN) + 4 * (lane >> 4);
    if (m >= g.M) return;
    const float sa = g.out == 2 ? 0.0f : g.sa[m];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < g.N) put(g, m, n + e, v[e], sa, g.out == 2 ? 0.0f : g.sw[n + e]);
}

// Which kernel takes a call.  Measured on MI355X, weights from HBM, us:
//   1 or 2 tokens: one channel tile a workgroup and 16 waves with rings of 3
//     / two tiles, 8 waves, rings of 3 / four, 8, 2 / one, 4, 5:
//       N = 4096, K = 4096    4.6 /  5.1 /  6.0 /  5.0   (3.7 TB/s of weights)
//       4096, 11008           8.9 /  9.4 / 13.2 /  8.9   (5.1)
//       5120, 5120            7.8 /  6.1 /  7.4 /  7.2   (4.3)
//       5120, 13824          18.2 / 15.1 / 22.4 / 17.3   (4.7)
//       8192, 8192           13.0 / 18.1 / 12.0 / 12.7   (5.6)
//       11008, 4096          11.2 / 11.6 /  9.6 / 11.9   (4.7)
//       11008, 8192          19.6 / 25.3 / 19.3 / 18.5   (4.9)
//       28672, 8192          44.6 / 55.2 / 47.3 / 40.7   (5.8)
//     so the first up to 4096 channels, the second up to 8192 but where rows
//     are a multiple of 8192 apart (its workgroups then meet on the same
//     memory channels), the third up to 16384 if k is short, else the fourth.
//   16 tokens: a ring of 16 waves does not fit with their 2 KiB of tokens a
//     unit; one tile and 8 waves with rings of 4 instead, 5.6 against 6.3 with
//     the fourth at 4096 x 4096; 11008 x 4096 9.7 with the third, 13.0 with
//     the fourth; 28672 x 8192 48.1 and 46.5.
//   24 tokens: few-token kernel 16.4 against 64 x 64 tiles 11.6 at N = 11008,
//     12.1 against 13.7 (4 k ranges) at N = 4096, K = 11008
//   40 tokens: 19.2 against 11.8; 14.7 against 14.2
//   64 tokens: 21.2 against 15.3; 17.9 against 14.6 (K = 11008); 8.3 against
//     9.6 (4096 x 4096)
//   k = 16384, against 64 x 64 tiles with their ranges of k: 24 tokens 13.0 and
//     11.7 at N = 2048, 40 tokens 11.5 and 10.2 at N = 1024; k = 11008, N = 2048,
//     24 tokens 8.0 and 10.8
// So the few-token kernel keeps up to 16 tokens, and up to 64 when there are
// too few channels for a tile on every CU and k is short enough.
// Tiles: 64 x 64, 64 x 128, 128 x 128, 256 x 256 with k ranges of 4096 take
// about max(11, 8.5 x), 14 ceil(x), max(18, 24 x) and (x <= 1: 40 + 17 x,
// else 57 ceil(x)) us for x = tiles / 256; the smallest is taken.
// (Short runs: 4096 x 11008 x 4096: 256 x 256 164 us, 128 x 128 227; 1024 x 4096 x 4096:
// 128 x 128 22.0, 256 x 256 40.6, 64 x 128 27.5; 512: 64 x 128 14.6, 64 x 64
// 16.4, 128 x 128 19.1; 256: 64 x 64 11.6, 64 x 128 13.5.)
// Too few 64 x 64 tiles for the CUs and a long k: the k range is split and
// joined by a second kernel, which costs about 4 us (M = 64, 4096 x 11008:
// 23.0 -> 14.6 us with 4 ranges; at K = 4096 and 64 tiles it gains nothing).
// Up to 8 ranges where there are few tiles: 64 x 1024 x 28672 47 us whole, 17.9
// with 4, 12.8 with 8; 128 x 256 x 16384 27.6, 12.1, 9.5.
enum { kTile64 = 5, kTile64x128 = 6, kTile128 = 7, kTile256 = 8 };

W8A8Plan w8a8_plan(const bitq_w8a8_desc& d) {
    W8A8Plan p{};
    p.splits = 1;
    if (d.M <= 16 || (d.M <= 64 && d.N <= 6144 && d.K <= (d.M <= 48 ? 12288 : 6144))) {
        p.kernel = (d.M + 15) / 16;
        return p;
    }
    auto tiles = [&](int64_t bm, int64_t bn) { return ((d.M + bm - 1) / bm) * ((d.N + bn - 1) / bn); };
    const int64_t t64 = tiles(64, 64);
    auto x = [&](int64_t bm, int64_t bn) { return static_cast<double>(tiles(bm, bn)) / 256; };
    auto up = [](double v) { return static_cast<double>(static_cast<int64_t>(v + 0.999999)); };
    const double x256 = x(256, 256);
    const double us[4] = {std::max(11.0, 8.5 * x(64, 64)), 14.0 * up(x(64, 128)), std::max(18.0, 24.0 * x(128, 128)),
                          x256 <= 1 ? 40 + 17 * x256 : 57 * up(x256)};
    p.kernel = kTile64;
    for (int i = 1; i < 4; ++i)
        if (us[i] < us[p.kernel - kTile64]) p.kernel = kTile64 + i;
    if (p.kernel == kTile64 && t64 <= 128 && (d.K >= 6144 || (t64 <= 32 && d.K >= 4096))) {
        p.splits = static_cast<int>(std::min<int64_t>({8, 256 / t64, d.K / 1024}));
        p.ws_bytes = static_cast<size_t>(p.splits) * t64 * 64 * 64 * 4;
    }
    return p;
}

template <int TT, int NB, int KW, int NS, int TC = 2 * TT>
static int launch_few(const GemmArgs& g, hipStream_t st) {
    hipLaunchKernelGGL((w8a8_few_kernel<TT, NB, KW, NS, TC>), dim3(static_cast<unsigned>((g.N + 16 * NB - 1) / (16 * NB))),
                       dim3(64 * KW), 0, st, g);
    return static_cast<int>(hipGetLastError());
}

template <int BM, int BN, int WM, int WN, int NS, int KSUB>
static int launch_tile(const GemmArgs& g, int splits, void* ws, hipStream_t st) {
    const int tm = (g.M + BM - 1) / BM, tn = (g.N + BN - 1) / BN;
    const int kper = ((g.K + splits - 1) / splits + 127) / 128 * 128;
    constexpr int lds = NS * KSUB * (BM + BN) * 64;
    auto kern = w8a8_tile_kernel<BM, BN, WM, WN, NS, KSUB>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return static_cast<int>(e);
    }
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tm) * tn * splits), dim3(64 * (BM / WM) * (BN / WN)), lds, st, g, tm, tn,
                       splits, kper, static_cast<int*>(ws));
    if (splits > 1)
        hipLaunchKernelGGL((w8a8_join_kernel<BM, BN, WM, WN>), dim3(static_cast<unsigned>(tm) * tn * (BM * BN / 1024)), dim3(256), 0,
                           st, g, tm, tn, splits, static_cast<const int*>(ws));
    return static_cast<int>(hipGetLastError());
}

int launch_gemm_w8a8(const bitq_w8a8_desc& d, const W8A8Plan& plan, const void* a, const float* sa, const void* w,
                     const float* sw, void* y, void* ws, void* stream) {
    const GemmArgs g{static_cast<const int8_t*>(a), static_cast<const int8_t*>(w), sa, sw, y, d.lda, d.ldw, d.ldy,
                     d.M, d.N, d.K, (d.flags & BITQ_F_ACC_INT32) ? 2 : d.y_dtype == BITQ_DT_BF16 ? 1 : 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    switch (plan.kernel) {
        case 1:
            if (d.N <= 4096) return d.M <= 8 ? launch_few<1, 1, 16, 3, 1>(g, st) : launch_few<1, 1, 8, 4>(g, st);
            if (d.N <= 8192 && d.ldw % 8192) return launch_few<1, 2, 8, 3>(g, st);
            if (d.N > 8192 && d.N <= 16384 && d.K <= 6144) return launch_few<1, 4, 8, 2>(g, st);
            return launch_few<1, 1, 4, 5>(g, st);
        case 2: return launch_few<2, 1, 8, 3>(g, st);
        case 3: return launch_few<3, 1, 8, 2>(g, st);
        case 4: return launch_few<4, 1, 8, 2>(g, st);
        case kTile64: return launch_tile<64, 64, 32, 32, 5, 2>(g, plan.splits, ws, st);
        case kTile64x128: return launch_tile<64, 128, 32, 64, 4, 2>(g, 1, ws, st);
        case kTile128: return launch_tile<128, 128, 64, 64, 5, 1>(g, 1, ws, st);
        default: return launch_tile<256, 256, 128, 64, 4, 1>(g, 1, ws, st);
    }
}

}  // namespace bitq
