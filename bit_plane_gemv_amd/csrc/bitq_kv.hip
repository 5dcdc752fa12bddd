// Paged key-value cache of libbitq: the planning kernel (page tables and slot
// maps from the requests' lengths) and the cache write.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "bitq_device.h"

namespace bitq {

// ================================================================== planning
// With held = ceil(old / page) and need = ceil(new / page), a request that
// grows takes need - held pages from the ring's head and gets new - old
// slots; one that shrinks puts held - need pages at the ring's end.  All of
// it follows from three prefix sums over the requests (tokens, pages taken,
// pages given back), so the kernel needs no communication between
// workgroups: each one computes the sums for all requests (at most 8192
// lengths, read from L2) into LDS, and then writes its share of the outputs,
// finding the request of an output by binary search in the sums.  A slot in
// a page taken by this very step is computed from the ring, not read from
// the table, which another workgroup may not have written yet.  The first
// token_groups workgroups write lengths, starts and slots, the others move
// pages.
//
// The sums saturate at 2^32 - 1 (saturating addition of counts is
// associative, so a scan of it is exact up to there, and every limit that a
// sum is compared with is below 2^29).
//
// Bound by latency: two dependent loads, the scan and one search.  64
// requests of one new token each 4.0 us, 1024 requests with 65536 new tokens
// (0.8 MB written) 7.2 us.
struct PlanOut {
    int32_t *state, *len, *start, *slot, *req, *pos;
};

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive sums over the workgroup of three values per thread (in thread
// order), with the total of each in tot.  s_w: a place for each wave.
__device__ __forceinline__ void block_scan3(uint32_t (&v)[3], uint32_t (&tot)[3], uint32_t (*s_w)[16]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const uint32_t t = __shfl_up(v[j], o, 64);
            v[j] = lane >= o ? add_sat(v[j], t) : v[j];
        }
    }
    __syncthreads();  // (the last round's reads of s_w are done)
    if (lane == 63) {
#pragma unroll
        for (int j = 0; j < 3; ++j) s_w[j][wave] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) {  // (all 16 places, read together; those past the last wave hold 0)
        uint32_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const uint32_t t = s_w[j][w];
            before = w < wave ? add_sat(before, t) : before;
            all = add_sat(all, t);
        }
        v[j] = add_sat(v[j], before);
        tot[j] = all;
    }
}

// First index i in [0, n) with a[i] > x (n if none); a ascending.
__device__ __forceinline__ int first_above(const uint32_t* a, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ __launch_bounds__(1024) void kv_plan_kernel(const int32_t* __restrict__ old_len,
                                                       const int32_t* __restrict__ new_len, int R, int page_shift,
                                                       int table_stride, int cap, int T, int32_t* ring,
                                                       const int32_t* __restrict__ state, int32_t* table, PlanOut out,
                                                       int token_groups) {
    extern __shared__ uint32_t s_mem[];
    uint32_t* s_tok = s_mem;                                        // [R] inclusive sums: new tokens,
    uint32_t* s_pop = s_mem + R;                                    //     pages taken,
    uint32_t* s_push = s_mem + 2 * R;                               //     pages given back
    int32_t* s_old = reinterpret_cast<int32_t*>(s_mem + 3 * R);     // lengths before
    __shared__ __align__(16) uint32_t s_w[3][16];
    __shared__ int s_refused;
    const int tid = threadIdx.x, nth = blockDim.x;
    const int64_t most = static_cast<int64_t>(table_stride) << page_shift;  // longest request the table holds (< 2^31)
    const uint32_t round = (1u << page_shift) - 1u;
    if (tid == 0) s_refused = 0;
    if (tid < 48) s_w[tid >> 4][tid & 15] = 0;
    int head = state[0] % cap;
    const int count = min(max(state[1], 0), cap);
    if (head < 0) head += cap;
    auto pages = [&](int len) { return static_cast<int>((static_cast<uint32_t>(len) + round) >> page_shift); };  // len >= 0
    auto in_ring = [&](uint32_t p) {  // place head + p of the ring, p < 2 cap
        const uint32_t i = (static_cast<uint32_t>(head) + p) % static_cast<uint32_t>(cap);
        return static_cast<int>(i);
    };

    // ---- the sums.  Refusals: the sums of a request count what every
    // earlier request asked for, and a growing request asks for at least one
    // token; so once one does not fit, no later one does, and the requests
    // served are those whose inclusive sums fit.
    uint32_t carry[3] = {0, 0, 0};           // asked for so far: tokens, pages; given back
    uint32_t served_tok = 0, served_pop = 0; // the largest sums of requests served
    constexpr uint32_t kRefused = 0xFFFFFFFFu;
    for (int r0 = 0; r0 < R; r0 += nth) {
        const int r = r0 + tid;
        int o = 0, n = 0;
        if (r < R) {
            o = old_len[r];
            n = new_len[r];
            s_old[r] = o;
        }
        const bool fits = o >= 0 && n >= 0 && o <= most && n <= most;
        const int held = fits ? pages(o) : 0, need = fits ? pages(n) : 0;
        const bool grow = fits && n > o;
        uint32_t v[3] = {grow ? static_cast<uint32_t>(n - o) : 0u, grow ? static_cast<uint32_t>(need - held) : 0u,
                         fits && n < o ? static_cast<uint32_t>(held - need) : 0u}, tot[3];
        block_scan3(v, tot, s_w);
        const uint32_t tok = add_sat(carry[0], v[0]), pop = add_sat(carry[1], v[1]);
        const bool given = grow && tok <= static_cast<uint32_t>(T) && pop <= static_cast<uint32_t>(count);
        if (given) {
            served_tok = tok;
            served_pop = pop;
        }
        const bool refused = r < R && (!fits || (grow && !given));
        if (r < R) {
            s_tok[r] = grow && !given ? kRefused : min(tok, kRefused - 1u);  // (settled below)
            s_pop[r] = pop;
            s_push[r] = add_sat(carry[2], v[2]);
        }
        if (blockIdx.x == 0 && refused) atomicAdd(&s_refused, 1);
#pragma unroll
        for (int j = 0; j < 3; ++j) carry[j] = add_sat(carry[j], tot[j]);
    }
    // totals served: the largest over the workgroup
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        served_tok = max(served_tok, __shfl_xor(served_tok, o, 64));
        served_pop = max(served_pop, __shfl_xor(served_pop, o, 64));
    }
    __syncthreads();
    if ((tid & 63) == 0) {
        s_w[0][tid >> 6] = served_tok;
        s_w[1][tid >> 6] = served_pop;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        served_tok = max(served_tok, s_w[0][w]);
        served_pop = max(served_pop, s_w[1][w]);
    }
    const uint32_t pushed = min(carry[2], static_cast<uint32_t>(cap - count));

    // ---- refused requests take no tokens and no pages: from the first one
    // on the sums are the served totals
    const int groups = token_groups, bid = blockIdx.x;
    for (int r = tid; r < R; r += nth) {
        const bool refused = s_tok[r] == kRefused;
        s_tok[r] = min(s_tok[r], served_tok);
        s_pop[r] = min(s_pop[r], served_pop);
        if (bid < groups && r % groups == bid) {
            const int o = s_old[r], n = new_len[r];
            const bool fits = o >= 0 && n >= 0 && o <= most && n <= most;
            out.len[r] = fits && !refused ? n : o;
        }
    }
    __syncthreads();
    if (bid < groups) {
        const int gid = bid * nth + tid, step = groups * nth;
        for (int r = gid; r <= R; r += step) out.start[r] = r == 0 ? 0 : static_cast<int>(s_tok[r - 1]);
        if (gid == 0) {
            out.state[0] = in_ring(served_pop);
            out.state[1] = count - static_cast<int>(served_pop) + static_cast<int>(pushed);
            out.state[2] = static_cast<int>(served_tok);
            out.state[3] = s_refused;
        }
        // ---- the new tokens' slots
        for (int t = gid; t < T; t += step) {
            int slot = -1, req = -1, pos = -1;
            if (static_cast<uint32_t>(t) < served_tok) {
                req = first_above(s_tok, R, t);
                const int o = s_old[req];
                pos = o + t - static_cast<int>(req ? s_tok[req - 1] : 0u);
                const int j = pos >> page_shift, held = pages(o);
                const int pg = j < held ? table[static_cast<size_t>(req) * table_stride + j]
                                        : ring[in_ring((req ? s_pop[req - 1] : 0u) + static_cast<uint32_t>(j - held))];
                slot = static_cast<int>((static_cast<uint32_t>(pg) << page_shift) + (static_cast<uint32_t>(pos) & round));
            }
            out.slot[t] = slot;
            out.req[t] = req;
            out.pos[t] = pos;
        }
        return;
    }
    // ---- pages taken, and pages given back (to places of the ring that are
    // free now: none that is read for a page taken)
    const uint32_t gid = static_cast<uint32_t>(bid - groups) * nth + tid, step = (gridDim.x - groups) * nth;
    for (uint32_t p = gid; p < served_pop; p += step) {
        const int r = first_above(s_pop, R, p);
        table[static_cast<size_t>(r) * table_stride + pages(s_old[r]) + (p - (r ? s_pop[r - 1] : 0u))] = ring[in_ring(p)];
    }
    for (uint32_t p = gid; p < pushed; p += step) {
        const int r = first_above(s_push, R, p);
        ring[in_ring(static_cast<uint32_t>(count) + p)] =
            table[static_cast<size_t>(r) * table_stride + pages(new_len[r]) + (p - (r ? s_push[r - 1] : 0u))];
    }
}

int launch_kv_plan(const bitq_kv_plan_desc& d, const int32_t* old_len, const int32_t* new_len, int32_t* ring,
                   const int32_t* state, int32_t* table, void* plan, void* stream) {
    const KvPlanLayout L = kv_plan_layout(d);
    uint8_t* b = static_cast<uint8_t*>(plan);
    auto at = [&](size_t off) { return reinterpret_cast<int32_t*>(b + off); };
    const PlanOut out{at(0), at(L.off_len), at(L.off_start), at(L.off_slot), at(L.off_req), at(L.off_pos)};
    const int shift = __builtin_ctz(static_cast<unsigned>(d.page));
    const int block = std::max(d.requests, d.tokens) <= 256 ? 256 : 1024;
    // one thread per token up to 256 workgroups (each repeats the sums), and
    // one per page moved, taken as up to 64 a request, up to 64 workgroups
    // (1024 requests, 72 of them finished: 11.6 us with 3, 6.9 with 64)
    const int groups = std::min(256, (std::max(d.requests, d.tokens) + block - 1) / block);
    const int movers = static_cast<int>(std::min<int64_t>(64, (int64_t(d.requests) * std::min(d.table_stride, 64) + block - 1) / block));
    const size_t lds = 4 * 4 * static_cast<size_t>(d.requests);
    static_assert(4 * 4 * 8192 <= 128 * 1024, "the sums of 8192 requests fit the LDS");
    if (lds > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kv_plan_kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return static_cast<int>(e);
    }
    hipLaunchKernelGGL(kv_plan_kernel, dim3(groups + movers), dim3(block), lds, static_cast<hipStream_t>(stream), old_len,
                       new_len, d.requests, shift, d.table_stride, d.ring, d.tokens, ring, state, table, out, groups);
    return static_cast<int>(hipGetLastError());
}

// =============================================================== cache write
// One thread takes 8 elements of a row: a 16-byte store of K.  V keeps 8
// tokens of an element together, so there a thread takes the 8 x 8 block of
// 8 consecutive slots: it reads 8 rows' 16 bytes and transposes in registers.
// Its 8 pieces of 16 bytes are 128 bytes apart from the next lane's; they are
// exchanged through LDS inside the wave, so that every store instruction
// writes 1 KB in a row (prompts of 4096 tokens, 32 heads of 128: 53 -> 38 us).
// TG = 8: a thread owns the groups that begin among its 8 tokens of the list
// (groups of consecutive slots are found from the slots, whatever their
// alignment to the list; at most one of them is whole); a group that is not
// whole, or TG = 1 (decode: every token in another page), stores single
// elements, which the L2 gathers.
// Int8 rows: the amax of a row is reduced over the threads that share it
// (LR = a power of two >= Dp / 8 lanes), then the arithmetic of the
// activation quantizer.
//
// Bound by HBM for long prompts (each element read and written once), by
// latency for decode.  Prompts of 4096 tokens, 32 heads of 128, bf16: 38 us,
// 134 MB at 3.5 TB/s (a copy of those bytes takes 26 us; K alone 14, at the
// copy's rate, V 22: its loads wait for the slots); into int8 rows 33.5 us (one
// prompt; into bf16 33.4).  64 tokens of 8 heads: 3.8 us.
//
// 8 elements of a row as loaded (converted where they are used: 8 rows of
// bf16 then take 32 registers).
template <int XDT>
struct Raw8 {
    uint4 a[XDT == BITQ_DT_F32 ? 2 : 1];
    __device__ __forceinline__ float operator[](int e) const {
        const uint4 q = a[XDT == BITQ_DT_F32 ? e >> 2 : 0];
        const int w = XDT == BITQ_DT_F32 ? e & 3 : e >> 1;
        const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
        if (XDT == BITQ_DT_F32) return __uint_as_float(u);
        return __uint_as_float((e & 1) ? u & 0xFFFF0000u : u << 16);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (*this)[e];
    }
    // elements i .. i + 7 of x, the first n present; vec: all 8, 16-byte aligned
    __device__ __forceinline__ void load(const void* x, int64_t i, int n, bool vec) {
        constexpr int last = XDT == BITQ_DT_F32 ? 1 : 0;
        if (vec) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + i * (XDT == BITQ_DT_F32 ? 4 : 2));
            a[0] = p[0];
            if (XDT == BITQ_DT_F32) a[last] = p[1];
        } else {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] = 0;
                if (e < n) u[e] = XDT == BITQ_DT_F32 ? static_cast<const uint32_t*>(x)[i + e] : static_cast<const uint16_t*>(x)[i + e];
            }
            if (XDT == BITQ_DT_F32) {
                a[0] = make_uint4(u[0], u[1], u[2], u[3]);
                a[last] = make_uint4(u[4], u[5], u[6], u[7]);
            } else {
                a[0] = make_uint4(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
            }
        }
    }
};

// Scale of a row from this thread's 8 elements (LR lanes share the row), and its codes in place.  The amax is the
// largest of the magnitudes' bits, so NaN passes as the largest of all; a product that is NaN (an infinity or NaN in the
// row; a zero where 127 / amax overflows) has the code 0.
__device__ __forceinline__ float row_codes(float (&v)[8], int LR) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(fabsf(v[e])));
    for (int o = 1; o < LR; o <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(m, o, 64)));
    const float a = __uint_as_float(m);
    const float s = a > 0.0f ? __fdiv_rn(127.0f, a) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], s);
    if (!(a < INFINITY && s < INFINITY)) {  // (a branch that rows of ordinary numbers skip: 8 selects fewer)
        asm volatile("");
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] == v[e] ? v[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(rintf(v[e]), -127.0f), 127.0f);
    return __fdiv_rn(a, 127.0f);
}

__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return bf16_bits(a) | (static_cast<uint32_t>(bf16_bits(b)) << 16);
}
__device__ __forceinline__ uint32_t code_quad(float a, float b, float c, float d) {
    return (static_cast<uint32_t>(static_cast<int>(a)) & 255u) | ((static_cast<uint32_t>(static_cast<int>(b)) & 255u) << 8) |
           ((static_cast<uint32_t>(static_cast<int>(c)) & 255u) << 16) | (static_cast<uint32_t>(static_cast<int>(d)) << 24);
}
template <int KVT>
__device__ __forceinline__ void store8(void* base, size_t i, const float (&v)[8]) {  // i: element, a multiple of 8
    if constexpr (KVT == BITQ_KV_BF16)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
            make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    else
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + i) =
            make_uint2(code_quad(v[0], v[1], v[2], v[3]), code_quad(v[4], v[5], v[6], v[7]));
}
template <int KVT>
__device__ __forceinline__ void store1(void* base, size_t i, float v) {
    if constexpr (KVT == BITQ_KV_BF16) static_cast<uint16_t*>(base)[i] = bf16_bits(v);
    else static_cast<int8_t*>(base)[i] = static_cast<int8_t>(static_cast<int>(v));
}

struct WriteArgs {
    const void *k, *v;
    int64_t ks, vs;  // token strides
    const int32_t* slots;
    uint8_t* cache;
    size_t off_v, off_ks, off_vs;
    int tokens, heads, D, Dp, page_shift, nslots;
    bool vec_k, vec_v;
};

// Grid (thread blocks of 256 lanes, 2): blockIdx.y = 0 K, 1 V.  Thread =
// (token group, head, lane of the row), the lanes of a row contiguous.
template <int XDT, int KVT, int TG>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a, int LR, int lr_shift) {
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int c = static_cast<int>(gid & (LR - 1));  // 8-element chunk of the row
    const int64_t gh = gid >> lr_shift;
    const int64_t grp = gh / a.heads;
    const int h = static_cast<int>(gh - grp * a.heads);
    const int64_t t0 = grp * TG;
    // (the lanes of a row leave together: the shuffles below stay inside them;
    // V with TG = 8 needs every lane of the wave)
    if (t0 >= a.tokens && (TG == 1 || blockIdx.y == 0)) return;
    const int nt = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(TG), a.tokens - t0)));
    const int n = min(8, a.D - 8 * c);          // elements of the chunk (<= 0: padding or a spare lane)
    const bool live = 8 * c < a.Dp;
    const int P = 1 << a.page_shift;
    if (blockIdx.y == 0) {
        void* K = a.cache;
        float* sc = reinterpret_cast<float*>(a.cache + a.off_ks);
        Raw8<XDT> x[TG];
#pragma unroll
        for (int e = 0; e < TG; ++e)
            x[e].load(a.k, min(t0 + e, static_cast<int64_t>(a.tokens) - 1) * a.ks + static_cast<int64_t>(h) * a.D + 8 * c, n,
                      a.vec_k && n == 8);
#pragma unroll
        for (int e = 0; e < TG; ++e) {
            const int slot = a.slots[min(t0 + e, static_cast<int64_t>(a.tokens) - 1)];
            float d = 0.0f, v[8];
            x[e].get(v);
            if constexpr (KVT == BITQ_KV_INT8) d = row_codes(v, LR);
            if (e < nt && static_cast<uint32_t>(slot) < static_cast<uint32_t>(a.nslots)) {
                const size_t row = (static_cast<size_t>(slot >> a.page_shift) * a.heads + h) * P + (slot & (P - 1));
                if (live) store8<KVT>(K, row * a.Dp + 8 * c, v);
                if (KVT == BITQ_KV_INT8 && c == 0) sc[row] = d;
            }
        }
        return;
    }
    void* V = a.cache + a.off_v;
    float* sc = reinterpret_cast<float*>(a.cache + a.off_vs);
    const int64_t vrow = static_cast<int64_t>(h) * a.D + 8 * c;
    // row of the pool (of this head) and element 0 of the 8-token group of a slot
    auto pool_row = [&](int slot) { return (static_cast<size_t>(slot >> a.page_shift) * a.heads + h) * P + (slot & (P - 1)); };
    auto group_at = [&](size_t row) { return (row >> 3) * a.Dp * 8; };  // (pages are whole groups)
    if constexpr (TG == 1) {
        Raw8<XDT> x;
        x.load(a.v, t0 * a.vs + vrow, n, a.vec_v && n == 8);
        float d = 0.0f, v[8];
        x.get(v);
        if constexpr (KVT == BITQ_KV_INT8) d = row_codes(v, LR);
        const int slot = a.slots[t0];
        if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(a.nslots)) return;
        const size_t row = pool_row(slot);
        if (KVT == BITQ_KV_INT8 && c == 0) sc[row] = d;
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) store1<KVT>(V, group_at(row) + (8 * c + i) * 8 + (row & 7), v[i]);
        }
    } else {
        // slots of tokens t0 - 7 .. t0 + 14 (-1 outside the list)
        int sb[7], sl[15];
#pragma unroll
        for (int e = 0; e < 7; ++e) sb[e] = a.slots[min(max(t0 - 1 - e, static_cast<int64_t>(0)), static_cast<int64_t>(a.tokens) - 1)];
#pragma unroll
        for (int e = 0; e < 15; ++e) sl[e] = a.slots[min(t0 + e, static_cast<int64_t>(a.tokens) - 1)];
        // (unconditional loads, issued together; selected afterwards)
#pragma unroll
        for (int e = 0; e < 7; ++e) sb[e] = t0 - 1 - e >= 0 && t0 - 1 - e < a.tokens ? sb[e] : -1;
#pragma unroll
        for (int e = 0; e < 15; ++e) sl[e] = t0 + e < a.tokens ? sl[e] : -1;
        auto inside = [&](int s) { return static_cast<uint32_t>(s) < static_cast<uint32_t>(a.nslots); };
        int whole = -1, wslot = -1;  // token (of the 8) at which a whole group begins, its slot
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            bool w = inside(sl[f]) && (sl[f] & 7) == 0;
#pragma unroll
            for (int e = 1; e < 8; ++e) w = w && sl[f + e] == sl[f] + e;
            whole = w ? f : whole;
            wslot = w ? sl[f] : wslot;
        }
        // tokens (of the 8) that belong to a whole group begun among the 7
        // before them: its owner stores them
        int back = 0, fore = 0;  // consecutive slots before and after the first token's
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            back = back == e && sb[e] == sl[0] - 1 - e ? e + 1 : back;
            fore = fore == e && sl[e + 1] == sl[0] + 1 + e ? e + 1 : fore;
        }
        const int in0 = sl[0] & 7;
        const int owned = inside(sl[0]) && in0 > 0 && back >= in0 && fore >= 7 - in0 ? 8 - in0 : 0;
        using Piece = typename std::conditional<KVT == BITQ_KV_BF16, uint4, uint2>::type;  // 8 tokens of an element
        __shared__ Piece s_x[4][512];
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const size_t wrow = whole >= 0 ? pool_row(wslot) : 0;
        if (whole >= 0) {
            Raw8<XDT> x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e].load(a.v, (t0 + whole + e) * a.vs + vrow, n, a.vec_v && n == 8);
            if constexpr (KVT == BITQ_KV_INT8) {  // codes in place of the elements
                float v[8][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e].get(v[e]);
                    const float d = row_codes(v[e], LR);
                    if (c == 0) sc[wrow + e] = d;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w[8] = {v[0][i], v[1][i], v[2][i], v[3][i], v[4][i], v[5][i], v[6][i], v[7][i]};
                    store8<KVT>(s_x[wave], (8 * lane + (i ^ (lane & 7))) * 8, w);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // element 8 c + i of the lane's row
                    const float w[8] = {x[0][i], x[1][i], x[2][i], x[3][i], x[4][i], x[5][i], x[6][i], x[7][i]};
                    store8<KVT>(s_x[wave], (8 * lane + (i ^ (lane & 7))) * 8, w);
                }
            }
        }
        asm volatile("" ::: "memory");  // (LDS operations of a wave keep their order)
        // the wave's rows, 64 pieces at a time: piece q is element q % (8 LR)
        // of the row of lanes (q / 8 LR) LR ..
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int q = 64 * k + lane, src = (q >> (lr_shift + 3)) << lr_shift, e = q & (8 * LR - 1);
            const int has = __shfl(whole, src, 64);
            const uint32_t lo = __shfl(static_cast<uint32_t>(wrow), src, 64);
            const uint32_t hi = __shfl(static_cast<uint32_t>(wrow >> 32), src, 64);
            const size_t row = (static_cast<size_t>(hi) << 32) | lo;
            const Piece x = s_x[wave][(q & ~7) | ((q & 7) ^ ((q >> 3) & 7))];
            if (has >= 0 && e < a.Dp) reinterpret_cast<Piece*>(V)[(row >> 3) * a.Dp + e] = x;
        }
        // what is not part of a whole group: single elements (the whole group
        // that begins here reaches past the 8 tokens)
        bool store[8], some = false;
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            store[f] = f >= owned && f < nt && inside(sl[f]) && !(whole >= 0 && f >= whole);
            some = some || store[f];
        }
        if (!__any(some)) return;
        Raw8<XDT> x[8];
#pragma unroll
        for (int f = 0; f < 8; ++f)
            x[f].load(a.v, min(t0 + f, static_cast<int64_t>(a.tokens) - 1) * a.vs + vrow, n, a.vec_v && n == 8);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            float d = 0.0f, v[8];
            x[f].get(v);
            if constexpr (KVT == BITQ_KV_INT8) d = row_codes(v, LR);
            if (store[f]) {
                const size_t row = pool_row(sl[f]);
                if (KVT == BITQ_KV_INT8 && c == 0) sc[row] = d;
                if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) store1<KVT>(V, group_at(row) + (8 * c + i) * 8 + (row & 7), v[i]);
                }
            }
        }
    }
}

template <int XDT, int KVT>
static void launch_write(const WriteArgs& a, hipStream_t st) {
    int LR = 4, shift = 2;
    while (8 * LR < a.Dp) {
        LR *= 2;
        ++shift;
    }
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.heads;
    // 8 tokens per thread once single tokens would give more than 2^17
    // threads.  Measured, bf16, runs of 100 slots (single slots), us with 1 / 8
    // tokens: 2^16 threads 5.3 / 10.3 (7.2 / 14.9), 2^17 8.9 / 9.5 (10.6 /
    // 17.6), 2^18 15.4 / 10.7 (17.3 / 21.9), 2^20 50.5 / 21.4 (78 / 81).
    if (rows * LR <= (1 << 17)) {
        const dim3 grid(static_cast<unsigned>((rows * LR + 255) / 256), 2);
        hipLaunchKernelGGL((kv_write_kernel<XDT, KVT, 1>), grid, dim3(256), 0, st, a, LR, shift);
    } else {
        const int64_t groups = (static_cast<int64_t>(a.tokens) + 7) / 8 * a.heads;
        const dim3 grid(static_cast<unsigned>((groups * LR + 255) / 256), 2);
        hipLaunchKernelGGL((kv_write_kernel<XDT, KVT, 8>), grid, dim3(256), 0, st, a, LR, shift);
    }
}

int launch_kv_write(const bitq_kvdesc& kv, const void* k, const void* v, int x_dtype, int64_t ks, int64_t vs,
                    const int32_t* slots, int tokens, void* cache, void* stream) {
    const KvLayout L = kv_layout(kv);
    WriteArgs a{};
    a.k = k;
    a.v = v;
    a.ks = ks;
    a.vs = vs;
    a.slots = slots;
    a.cache = static_cast<uint8_t*>(cache);
    a.off_v = L.off_v;
    a.off_ks = L.off_ks;
    a.off_vs = L.off_vs;
    a.tokens = tokens;
    a.heads = kv.kv_heads;
    a.D = kv.head_dim;
    a.Dp = L.Dp;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(kv.page));
    a.nslots = kv.pages * kv.page;
    // rows whose every 8-element chunk is 16-byte aligned
    const int e = x_dtype == BITQ_DT_F32 ? 4 : 2, per = 16 / e;
    a.vec_k = aligned(k, 16) && ks % per == 0 && kv.head_dim % per == 0;
    a.vec_v = aligned(v, 16) && vs % per == 0 && kv.head_dim % per == 0;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (x_dtype == BITQ_DT_F32) {
        if (kv.dtype == BITQ_KV_BF16) launch_write<BITQ_DT_F32, BITQ_KV_BF16>(a, st);
        else launch_write<BITQ_DT_F32, BITQ_KV_INT8>(a, st);
    } else {
        if (kv.dtype == BITQ_KV_BF16) launch_write<BITQ_DT_BF16, BITQ_KV_BF16>(a, st);
        else launch_write<BITQ_DT_BF16, BITQ_KV_INT8>(a, st);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
