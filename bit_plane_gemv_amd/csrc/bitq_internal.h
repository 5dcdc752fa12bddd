// Internal declarations shared by the host side (bitq_host.cpp) and the HIP
// kernels (bitq_kernels.hip).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/bitq.h"
#include "../../include/bitq_ctx.h"
#include "../../include/bitq_lm.h"

namespace bitq {

constexpr int kRowTile = 64;      // rows per tile = lanes per wave
constexpr int kKBlock = 128;      // inputs per k block = 4 words per row
constexpr int kHeaderBytes = 256;
constexpr uint32_t kMagic = 0x51544942u;
constexpr int kHdrHBound = 72;    // header: f32 [3] max_k |h_p[k]| (SIGN1: 1)
constexpr int kMaxFloatK = 63 * 8 * kKBlock;  // float formats: <= 63 splits of <= 8 k blocks
constexpr int kWholeRowGrid = 256;  // whole-row kernels: workgroups (one per CU of the MI355X)
// LDS a whole-row kernel's workgroup claims at least: more than half of a
// CU's 160 KB, so the 256 workgroups land on 256 distinct CUs
constexpr int kOneWgPerCuLds = 84 * 1024;
// HGF header fields: u64 off_c2, u32 rank, f32 alpha, f32 gate, f32 amax_a
constexpr int kHdrOffC2 = 88, kHdrRank = 96, kHdrAlpha = 100, kHdrGate = 104, kHdrAmaxA = 108;
constexpr int kMaxHgfK = 63 * 256;  // HGF: <= 63 runs of 256 inputs meet in one fixed-point word

// BVSR4 planes: nibble e (0..7) of a plane word holds the bitvector bits of
// input (e >> 1) + 4 (e & 1) of the word's 8 inputs (the order in which two
// words of 4 activation bytes split into nibble words most cheaply)
constexpr int bvsr_nibble_input(int e) { return (e >> 1) + 4 * (e & 1); }

// The calling thread's error text (bitq_last_error): set and return s; clear.
bitq_status fail(bitq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
bitq_status ok();
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Byte layout of a packed blob (see include/bitq.h, "Packed blob layout").
struct BlobLayout {
    int64_t Np, Kp, P, Tn, Tb;
    size_t off_planes, planes_bytes;
    size_t off_c0, c0_bytes;
    size_t off_c1, c1_bytes;
    size_t off_c2, c2_bytes;  // HGF: B transposed (otherwise off_c2 = total, 0 bytes)
    size_t total;
};
BlobLayout blob_layout(const bitq_wdesc& d);

// Byte layout of an activation buffer (see bitq_quantize_act); rank > 0
// adds the HGF section h f32 [M][rank].
struct ActLayout {
    int64_t M, K, Kp, Kw;
    size_t off_planes, off_S, off_q, off_qm, off_d, off_amax, off_h, total;
};
// Rows longer than this get their amax from a separate pass (act_amax_kernel)
// instead of every workgroup of the quantizer reading the whole row.
constexpr int kAmaxOnePassK = 16384;
ActLayout act_layout(int M, int K, int rank = 0);

// Byte layout of a binary activation buffer (see bitq_binarize_act).
struct BinActLayout {
    int64_t M, K, Kp, Kw;
    size_t off_beta, total;
};
BinActLayout binact_layout(int M, int K);

// How a GEMV/GEMM call is split over workgroups, and its workspace.
struct Plan {
    int waves_per_wg;      // 64-row waves per workgroup
    int rows_per_wg;       // 64 * waves_per_wg
    int row_groups;        // ceil(Np / rows_per_wg)
    int blocks_per_split;  // k blocks (128 inputs) per workgroup
    int splits;            // ceil((Kp/128) / blocks_per_split)
    int M;
    size_t off_partials;   // float formats: u64 [Np] split-k words (count + fixed-point sum)
    size_t ws_bytes;
    bool mfma;             // TERNARY/W2A8/WNAM, M >= mfma_min_tokens: the int8 matrix-core kernel
};
Plan make_plan(const bitq_wdesc& d, int M, bool fused = false);  // fused: BITQ_F_FUSE_QUANT
// The fused-quantizer GEMV with 16 rows per workgroup, and the BVSR4 GEMV
// of one token with 16 rows, take 8 waves (32 k-groups) instead of 4 when
// the k range has more than this many 128-input blocks: then 4 waves would
// leave 4 or more blocks per lane.  Measured: fused W2A8 4096x11008 6.96 ->
// 6.57 us, fused BVSR 28672x8192 27.95 -> 27.58 us, BVSR 28672x8192
// 26.33 -> 25.75 us; slower with 4096 inputs (fused W2A8 11008x4096 5.67 ->
// 5.95 us, fused ternary 4096x4096 3.65 -> 3.92 us) and for the other
// formats' two-launch GEMVs (W2A8 4096x11008 5.02 -> 5.43 us).
constexpr int kWideMinBlocks = 48;

// Launch shape of the matrix-core kernel for M tokens: TT token tiles of 16,
// RS = kMfmaSubs (or 1, when the sub-tiles do not outnumber the workgroups)
// sub-tiles of 16 rows per pass of a workgroup, KW waves over
// k, CH k blocks whose loads a wave issues together; grid = one workgroup
// per CU (at most one per sub-tile), of 64 KW lanes.
constexpr int kMfmaSubs = 3;
struct MfmaShape {
    int TT, RS, KW, CH;
    int grid, block;
};
MfmaShape mfma_shape(const bitq_wdesc& d, int M);

// Workgroups and lanes per workgroup of the kernel a bitq_gemv /
// bitq_gemm_smallM call launches (x_dtype and flags as in that call).
struct LaunchShape {
    int grid, block;
};
LaunchShape launch_shape(const bitq_wdesc& d, int M, int x_dtype, uint32_t flags);
// Workgroups of the AND+popcount / XNOR kernels: 64/RG row groups per 64-row
// tile, tiles dealt round-robin to the 8 XCDs (padded to whole rounds).
inline int xcd_row_groups(int64_t tiles, int RG) { return static_cast<int>(8 * (64 / RG) * ((tiles + 7) / 8)); }
// Tokens from which TERNARY, W2A8 and WNAM run on the int8 matrix cores
// (measured on W2A8 11008x4096: 6.2 us at 2 and 3 tokens against 7.0 and
// 9.0 us on the VALU; ternary 4096x4096: 4.8 us at 2 and 3 tokens against
// 4.1 and 5.0 us).  0 for the formats that stay on the VALU.
inline int mfma_min_tokens(int fmt) {
    if (fmt == BITQ_W2A8 || fmt == BITQ_WNAM) return 2;
    if (fmt == BITQ_TERNARY) return 3;
    return 0;
}
constexpr int kMaxFusedK = 16384;    // BITQ_F_FUSE_QUANT: whole k range in one round of the kernel
constexpr int kLaunchNotBuilt = -1;  // launcher: no kernel built for this combination

// Kernel launchers (bitq_act.hip, bitq_sign.hip, bitq_bits.hip, bitq_mfma.hip,
// bitq_xnor.hip).  Arguments are already validated.
// Each returns hipSuccess or the HIP error code of the launch.
int launch_quantize_act(const void* x, int x_dtype, int M, int K, int abits, void* act, void* stream);
int launch_gemv_float(const bitq_wdesc& d, const Plan& plan, const void* w, const void* x,
                      int x_dtype, float* y, void* ws, void* stream);
// Small-M GEMM on the int8 matrix cores (plans with mfma set).
int launch_gemm_mfma(const bitq_wdesc& d, const void* w, const void* act, int M, float* y, uint32_t flags,
                     void* stream);
int launch_gemv_int(const bitq_wdesc& d, const Plan& plan, const void* w, const void* act,
                    int M, float* y, void* ws, uint32_t flags, void* stream);
// Fused activation quantizer + GEMV, one token, raw x (bf16 or fp32); returns
// kLaunchNotBuilt when the plan has no such kernel.
int launch_gemv_fused(const bitq_wdesc& d, const Plan& plan, const void* w, const void* x, int x_dtype, float* y,
                      void* stream);
int launch_quantize_act_hgf(const void* x, int x_dtype, int M, int K, int rank, const void* w, const BlobLayout& L,
                            void* act, void* ws, void* stream);
// The HGF activation step with its workspace in the library's static device
// scratch (bitq_quantize_act_hgf_noalloc): at most kNoAllocScratchWords
// 64-bit words (M * rank), allocates nothing.
constexpr int kNoAllocScratchWords = 64 * 64;
int launch_quantize_act_hgf_noalloc(const void* x, int x_dtype, int M, int K, int rank, const void* w,
                                    const BlobLayout& L, void* act, void* stream);
int launch_binarize_act(const void* x, int x_dtype, int M, int K, void* act, void* stream);
int launch_gemv_xnor(const bitq_wdesc& d, const void* w, const void* act, int M, float* y, uint32_t flags,
                     void* stream);

// Measurement context kernels (bitq_ctx.hip); arguments already validated.
int launch_ctx_empty(int grid, void* stream);
int launch_ctx_stream(const void* src, size_t bytes, int grid, float* out, int nout, void* stream);
int launch_ctx_spin(int microseconds, void* stream);

// ------------------------------------------------- operators of bitq_lm.h
// Byte layout of a cache buffer; strides in elements of the rows.
struct KvLayout {
    int Dp;
    size_t off_v, off_ks, off_vs, total;
};
inline KvLayout kv_layout(const bitq_kvdesc& kv) {
    KvLayout L{};
    L.Dp = static_cast<int>(round_up(kv.head_dim, 32));
    const size_t rows = static_cast<size_t>(kv.pages) * kv.page * kv.kv_heads;
    const size_t sec = align256(rows * L.Dp * (kv.dtype == BITQ_KV_BF16 ? 2 : 1));
    L.off_v = sec;
    L.off_ks = 2 * sec;
    L.off_vs = L.off_ks + (kv.dtype == BITQ_KV_INT8 ? align256(rows * 4) : 0);
    L.total = L.off_vs + (kv.dtype == BITQ_KV_INT8 ? align256(rows * 4) : 0);
    return L;
}

// Byte layout of a plan buffer.
struct KvPlanLayout {
    size_t off_len, off_start, off_slot, off_req, off_pos, total;
};
inline KvPlanLayout kv_plan_layout(const bitq_kv_plan_desc& d) {
    KvPlanLayout L{};
    L.off_len = 256;
    L.off_start = L.off_len + align256(4 * static_cast<size_t>(d.requests));
    L.off_slot = L.off_start + align256(4 * (static_cast<size_t>(d.requests) + 1));
    const size_t t = align256(4 * static_cast<size_t>(d.tokens));
    L.off_req = L.off_slot + t;
    L.off_pos = L.off_req + t;
    L.total = L.off_pos + t;
    return L;
}

// How a paged attention call is split over workgroups (bitq_attn.hip).
constexpr int kAttnWaves = 4;                    // waves per workgroup
constexpr int kAttnUnit = 32 * kAttnWaves;       // tokens a workgroup takes per pass
constexpr int kAttnMaxSplitRequests = 4096;      // the split kernel keeps their prefix sums in LDS
// Workgroups per CU of the kernel for rows of 32 nc elements (q32: fp32 q):
// as many as hide the memory's latency, and no more than registers allow
// without spilling in the loop.  Measured, 64 ragged requests of up to
// 4096 tokens, 64 heads on 8, us: bf16 rows of 96 88 with 2 and 91 with 3,
// int8 rows of 128 71 with 2 and 74 with 3, of 64 42 with 4 and 46 with 3;
// bf16 rows of 64, 2 requests of 30000 tokens, 30.7 with 3 and 33.1 with 4.
constexpr int attn_groups_per_cu(int kv_dtype, int nc, bool q32) {
    return kv_dtype == BITQ_KV_INT8 ? (nc <= 2 ? 4 : nc == 3 ? 3 : nc <= (q32 ? 6 : 7) ? 2 : 1)
                                    : (nc <= 2 ? 3 : nc <= (q32 ? 5 : 6) ? 2 : 1);
}
struct AttnPlan {
    int Dp, group, tiles;  // padded row, query heads per key-value head, 16-head tiles of them
    int items;             // requests x key-value heads x tiles
    int grid;              // workgroups of the main kernel
    int waves;             // and their waves
    bool split;            // tokens split over workgroups and joined by a second kernel
    size_t off_part, ws_bytes;
};
AttnPlan attn_plan(const bitq_attn_desc& d);

struct W8A8Plan {
    int kernel;            // which kernel (bitq_w8a8.hip)
    int splits;
    size_t ws_bytes;
};
W8A8Plan w8a8_plan(const bitq_w8a8_desc& d);

int launch_kv_plan(const bitq_kv_plan_desc& d, const int32_t* old_len, const int32_t* new_len, int32_t* ring,
                   const int32_t* state, int32_t* table, void* plan, void* stream);
int launch_kv_write(const bitq_kvdesc& kv, const void* k, const void* v, int x_dtype, int64_t ks, int64_t vs,
                    const int32_t* slots, int tokens, void* cache, void* stream);
int launch_paged_attn(const bitq_attn_desc& d, const AttnPlan& plan, const void* q, int64_t q_stride,
                      const void* cache, const int32_t* table, const int32_t* lens, void* out, float* lse, void* ws,
                      void* stream);
int launch_block_norm(const bitq_norm_desc& d, const void* u, const void* r, const void* post, const void* gate,
                      const void* pre, void* ro, void* h, float* dscale, void* stream);
int launch_gemm_w8a8(const bitq_w8a8_desc& d, const W8A8Plan& plan, const void* a, const float* sa, const void* w,
                     const float* sw, void* y, void* ws, void* stream);

// Device check (bitq_act.hip): is the current device a gfx950?
int current_device_is_gfx950(int* is_gfx950);

}  // namespace bitq
