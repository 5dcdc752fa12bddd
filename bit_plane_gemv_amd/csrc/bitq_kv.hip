// Paged key-value cache of libbitq: the planning kernel (page tables and slot
// maps from the requests' lengths) and the cache write.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitq_device.h"

namespace bitq {

// ================================================================== planning
// With held = ceil(old / page) and need = ceil(new / page), a request that
// grows takes need - held pages from the ring's head and gets new - old
// slots; one that shrinks puts held - need pages at the ring's end.  All of
// it follows from three prefix sums over the requests (pages taken, tokens,
// pages given back), so the kernel needs no communication between
// workgroups: each one computes the sums for all requests (at most 8192
// lengths, read from L2) into LDS, and then writes its share of the outputs,
// finding the request of an output by binary search in the sums.  A slot in
// a page taken by this very step is computed from the ring, not read from
// the table, which another workgroup may not have written yet.
//
// Bound by latency: two dependent loads, the scan and one search.
struct PlanOut {
    int32_t *state, *len, *start, *slot, *req, *pos;
};

// Inclusive sums over the workgroup of three values per thread (in thread
// order), with the total of each in tot.  s_w: 3 x waves.
__device__ __forceinline__ void block_scan3(int64_t (&v)[3], int64_t (&tot)[3], int64_t (*s_w)[16]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int64_t t = __shfl_up(v[j], o, 64);
            if (lane >= o) v[j] += t;
        }
    }
    __syncthreads();  // (the last round's reads of s_w are done)
    if (lane == 63) {
#pragma unroll
        for (int j = 0; j < 3; ++j) s_w[j][wave] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        int64_t before = 0, all = 0;
        for (int w = 0; w < waves; ++w) {
            const int64_t t = s_w[j][w];
            before += w < wave ? t : 0;
            all += t;
        }
        v[j] += before;
        tot[j] = all;
    }
}

// First index i in [0, n) with a[i] > x (n if none); a ascending.
__device__ __forceinline__ int first_above(const int32_t* a, int n, int x) {
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
                                                       const int32_t* __restrict__ state, int32_t* table, PlanOut out) {
    extern __shared__ int32_t s_mem[];
    int32_t* s_tok = s_mem;           // [R] inclusive sums: new tokens,
    int32_t* s_pop = s_mem + R;       //     pages taken,
    int32_t* s_push = s_mem + 2 * R;  //     pages given back
    __shared__ int64_t s_w[3][16];
    __shared__ int s_refused;
    const int tid = threadIdx.x, nth = blockDim.x;
    const int64_t most = static_cast<int64_t>(table_stride) << page_shift;  // longest request the table holds
    const int round = (1 << page_shift) - 1;
    if (tid == 0) s_refused = 0;
    int head = state[0] % cap, count = min(max(state[1], 0), cap);
    if (head < 0) head += cap;

    // ---- the sums.  Refusals: the sums of a request count what every
    // earlier request asked for, and a growing request asks for at least one
    // token; so once one does not fit, no later one does, and the requests
    // served are those whose inclusive sums fit.
    int64_t carry[3] = {0, 0, 0};          // asked for so far: tokens, pages; given back
    int served_tok = 0, served_pop = 0;    // (kept per thread: the largest served sums)
    for (int r0 = 0; r0 < R; r0 += nth) {
        const int r = r0 + tid;
        int o = 0, n = 0;
        if (r < R) {
            o = old_len[r];
            n = new_len[r];
        }
        const bool fits = o >= 0 && n >= 0 && o <= most && n <= most;
        const int held = fits ? static_cast<int>((static_cast<int64_t>(o) + round) >> page_shift) : 0;
        const int need = fits ? static_cast<int>((static_cast<int64_t>(n) + round) >> page_shift) : 0;
        const bool grow = fits && n > o;
        int64_t v[3] = {grow ? n - o : 0, grow ? need - held : 0, fits && n < o ? held - need : 0}, tot[3];
        block_scan3(v, tot, s_w);
        const int64_t tok = carry[0] + v[0], pop = carry[1] + v[1], push = carry[2] + v[2];
        const bool given = grow && tok <= T && pop <= count;
        if (given) {
            served_tok = static_cast<int>(tok);
            served_pop = static_cast<int>(pop);
        }
        if (r < R) {
            // refused requests are resolved below (their sums become the served totals)
            s_tok[r] = grow && !given ? -1 : static_cast<int>(min(tok, static_cast<int64_t>(INT32_MAX)));
            s_pop[r] = static_cast<int>(min(pop, static_cast<int64_t>(INT32_MAX)));
            s_push[r] = static_cast<int>(min(push, static_cast<int64_t>(INT32_MAX)));
            if (r < R && (!fits || (grow && !given)) && blockIdx.x == 0) atomicAdd(&s_refused, 1);
        }
        carry[0] += tot[0];
        carry[1] += tot[1];
        carry[2] += tot[2];
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
    for (int w = 0; w < (nth >> 6); ++w) {
        served_tok = max(served_tok, static_cast<int>(s_w[0][w]));
        served_pop = max(served_pop, static_cast<int>(s_w[1][w]));
    }
    const int pushed = static_cast<int>(min(carry[2], static_cast<int64_t>(cap - count)));

    // ---- lengths and starts; refused requests take no tokens and no pages
    for (int r = tid; r < R; r += nth) {
        const bool refused_grow = s_tok[r] < 0;
        s_tok[r] = refused_grow ? served_tok : min(s_tok[r], served_tok);
        s_pop[r] = refused_grow ? served_pop : min(s_pop[r], served_pop);
        if (r % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x)) {
            const int o = old_len[r], n = new_len[r];
            const bool fits = o >= 0 && n >= 0 && o <= most && n <= most;
            out.len[r] = fits && !refused_grow ? n : o;
        }
    }
    __syncthreads();
    const int gid = blockIdx.x * nth + tid, gstep = gridDim.x * nth;
    for (int r = gid; r <= R; r += gstep) out.start[r] = r == 0 ? 0 : s_tok[r - 1];
    if (gid == 0) {
        const int left = count - served_pop + pushed;
        out.state[0] = static_cast<int>((static_cast<int64_t>(head) + served_pop) % cap);
        out.state[1] = left;
        out.state[2] = served_tok;
        out.state[3] = s_refused;
    }

    // ---- the new tokens' slots
    for (int t = gid; t < T; t += gstep) {
        int slot = -1, req = -1, pos = -1;
        if (t < served_tok) {
            req = first_above(s_tok, R, t);
            const int o = old_len[req];
            pos = o + t - (req ? s_tok[req - 1] : 0);
            const int j = pos >> page_shift;
            const int held = static_cast<int>((static_cast<int64_t>(o) + round) >> page_shift);
            int pg;
            if (j < held) {
                pg = table[static_cast<size_t>(req) * table_stride + j];
            } else {
                const int64_t p = static_cast<int64_t>(head) + (req ? s_pop[req - 1] : 0) + (j - held);
                pg = ring[p % cap];
            }
            slot = static_cast<int>((static_cast<uint32_t>(pg) << page_shift) + (pos & round));
        }
        out.slot[t] = slot;
        out.req[t] = req;
        out.pos[t] = pos;
    }
    // ---- pages taken, and pages given back (places of the ring that are
    // free now: none that is read above)
    for (int p = gid; p < served_pop; p += gstep) {
        const int r = first_above(s_pop, R, p);
        const int held = static_cast<int>((static_cast<int64_t>(old_len[r]) + round) >> page_shift);
        table[static_cast<size_t>(r) * table_stride + held + p - (r ? s_pop[r - 1] : 0)] =
            ring[(static_cast<int64_t>(head) + p) % cap];
    }
    for (int p = gid; p < pushed; p += gstep) {
        const int r = first_above(s_push, R, p);
        const int need = static_cast<int>((static_cast<int64_t>(new_len[r]) + round) >> page_shift);
        ring[(static_cast<int64_t>(head) + count + p) % cap] =
            table[static_cast<size_t>(r) * table_stride + need + p - (r ? s_push[r - 1] : 0)];
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
    // one thread per token up to 256 workgroups; each repeats the sums
    const int grid = std::min(256, (std::max(d.requests, d.tokens) + block - 1) / block);
    const size_t lds = 3 * 4 * static_cast<size_t>(d.requests);
    static_assert(3 * 4 * 8192 <= 128 * 1024, "the sums of 8192 requests fit the LDS");
    if (lds > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kv_plan_kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return static_cast<int>(e);
    }
    hipLaunchKernelGGL(kv_plan_kernel, dim3(grid), dim3(block), lds, static_cast<hipStream_t>(stream), old_len, new_len,
                       d.requests, shift, d.table_stride, d.ring, d.tokens, ring, state, table, out);
    return static_cast<int>(hipGetLastError());
}

// =============================================================== cache write
// One thread takes 8 elements of a row: a 16-byte store of K.  V keeps 8
// tokens of an element together, so there a thread takes the 8 x 8 block of
// 8 consecutive tokens: it reads 8 rows' 16 bytes, transposes in registers
// and stores 8 x 16 bytes.  TG = 8 threads own the token groups that begin
// among their 8 tokens of the list (groups of consecutive slots are found
// from the slots, whatever their alignment to the list); a group that is not
// whole, or TG = 1 (decode: every token in another page), stores single
// elements, which the L2 gathers.
// Int8 rows: the amax of a row is reduced over the threads that share it
// (LR = a power of two >= Dp / 8 lanes), then the arithmetic of the
// activation quantizer.
//
// Bound by HBM for long prompts (each element read and written once), by
// latency for decode.
template <int XDT>
__device__ __forceinline__ void load8(const void* x, int64_t i, int n, bool vec, float (&v)[8]) {
    if (vec) {  // 16-byte aligned and whole
        if (XDT == BITQ_DT_F32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
            const float4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? act_at<XDT>(x, static_cast<size_t>(i + e)) : 0.0f;
    }
}

// Scale of a row from this thread's 8 elements (LR lanes share the row), and its codes in place.
__device__ __forceinline__ float row_codes(float (&v)[8], int LR) {
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(v[e]));
    for (int o = 1; o < LR; o <<= 1) a = fmaxf(a, __shfl_xor(a, o, 64));
    const float s = a > 0.0f ? __fdiv_rn(127.0f, a) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(rintf(__fmul_rn(v[e], s)), -127.0f), 127.0f);
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
    // (the lanes of a row leave together: the shuffles below stay inside them)
    if (t0 >= a.tokens) return;
    const int nt = static_cast<int>(min(static_cast<int64_t>(TG), a.tokens - t0));
    const int n = min(8, a.D - 8 * c);          // elements of the chunk (<= 0: padding or a spare lane)
    const bool live = 8 * c < a.Dp;
    const int P = 1 << a.page_shift;
    if (blockIdx.y == 0) {
        void* K = a.cache;
        float* sc = reinterpret_cast<float*>(a.cache + a.off_ks);
        float v[TG][8];
#pragma unroll
        for (int e = 0; e < TG; ++e)
            load8<XDT>(a.k, min(t0 + e, static_cast<int64_t>(a.tokens) - 1) * a.ks + static_cast<int64_t>(h) * a.D + 8 * c,
                       n, a.vec_k && n == 8, v[e]);
#pragma unroll
        for (int e = 0; e < TG; ++e) {
            if (e >= nt) break;
            const int slot = a.slots[t0 + e];
            float d = 0.0f;
            if constexpr (KVT == BITQ_KV_INT8) d = row_codes(v[e], LR);
            if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(a.nslots)) continue;
            const size_t row = (static_cast<size_t>(slot >> a.page_shift) * a.heads + h) * P + (slot & (P - 1));
            if (live) store8<KVT>(K, row * a.Dp + 8 * c, v[e]);
            if (KVT == BITQ_KV_INT8 && c == 0) sc[row] = d;
        }
        return;
    }
    void* V = a.cache + a.off_v;
    float* sc = reinterpret_cast<float*>(a.cache + a.off_vs);
    for (int f = 0; f < nt; ++f) {
        const int64_t t = t0 + f;
        const int slot = a.slots[t];
        if (TG > 1 && t > 0) {
            const int before = a.slots[t - 1];
            // token t continues the group of token t - 1 (taken with its first token)
            if (before >= 0 && slot == before + 1 && (slot & 7) != 0) {
                // ... unless that group is longer than this thread's reach back: groups have at most 8 tokens
                continue;
            }
        }
        // the group: consecutive slots up to a multiple of 8
        int m = 1;
        if (TG > 1) {
            const int most = 8 - (slot & 7);
            for (int e = 1; e < 8; ++e)
                if (m == e && e < most && t + e < a.tokens && a.slots[t + e] == slot + e) m = e + 1;
        }
        const bool in = static_cast<uint32_t>(slot) < static_cast<uint32_t>(a.nslots);
        const size_t page_head = static_cast<size_t>(slot >> a.page_shift) * a.heads + h;  // (used only if in)
        const int off = slot & (P - 1);
        const size_t at = (page_head * (P >> 3) + (off >> 3)) * a.Dp * 8;  // element 0 of the group
        if (TG > 1 && m == 8) {
            float v[8][8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                load8<XDT>(a.v, (t + e) * a.vs + static_cast<int64_t>(h) * a.D + 8 * c, n, a.vec_v && n == 8, v[e]);
            if constexpr (KVT == BITQ_KV_INT8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = row_codes(v[e], LR);
                    if (c == 0 && in) sc[page_head * P + off + e] = d;
                }
            }
            if (in && live) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w[8] = {v[0][i], v[1][i], v[2][i], v[3][i], v[4][i], v[5][i], v[6][i], v[7][i]};
                    store8<KVT>(V, at + (8 * c + i) * 8, w);
                }
            }
        } else {
            for (int e = 0; e < m; ++e) {
                float v[8];
                load8<XDT>(a.v, (t + e) * a.vs + static_cast<int64_t>(h) * a.D + 8 * c, n, a.vec_v && n == 8, v);
                if constexpr (KVT == BITQ_KV_INT8) {
                    const float d = row_codes(v, LR);
                    if (c == 0 && in) sc[page_head * P + off + e] = d;
                }
                if (in && live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) store1<KVT>(V, at + (8 * c + i) * 8 + ((off + e) & 7), v[i]);
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
    // 8 tokens per thread once single tokens would give more than 2^16 threads
    if (rows * LR <= (1 << 16)) {
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
