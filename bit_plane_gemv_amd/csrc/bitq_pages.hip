// Pages of the cache held by several requests: forking, cutting and freeing
// requests, compacting the pool, and copies of pages.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitq_device.h"

namespace bitq {

// Who holds what is found from the tables: every page has one word, the least
// of what the requests claim of it,
//   0              somebody holds it whole after the call
//   1 + key        requests end inside it; key = r of the one that had it (src =
//                  r), or R + r of the first that asks for it
//   kHeld          somebody held it before the call, nobody does after it
//   kNone          a free page
// A minimum does not depend on the order of its operands, and everything else
// follows from the words and from prefix sums (over the requests: page copies
// asked for; over the pool: pages given back, or held), so results are the same
// from run to run.  The phases need all of the one before:
//   clear the words - claims - decisions and sums - outputs.
// Small pools have their words in LDS and one workgroup goes through all of it;
// larger ones take a launch for each phase, with the words in the workspace.
constexpr uint32_t kNone = 0xFFFFFFFFu, kHeld = 0xFFFFFFFEu;
constexpr int kSeg = kPagesSegment;  // pages of the pool that a workgroup sums

struct PagesArgs {
    const int32_t *src, *keep, *len, *table, *state;
    int32_t *ring, *table_out;
    int32_t *o_state, *o_len, *o_frm, *o_to;
    uint32_t* words;   // [pool]
    int32_t* sums;     // [segments]: freed (fork) or held (compact) pages of each
    int32_t* fresh;    // fork: [R] the copy's page (-1: none)
    int32_t* rank;     // compact: [pool] a moved page's place in the list (else -1)
    int R, S, page_shift, pool, M;
};

struct Request {
    int src, keep, len;  // as taken: the request's own if what it asks for is refused
    bool refused;
};
__device__ __forceinline__ int held_len(const PagesArgs& a, int r) {
    const int64_t most = static_cast<int64_t>(a.S) << a.page_shift;  // (< 2^31)
    return min(max(a.len[r], 0), static_cast<int>(most));
}
__device__ __forceinline__ Request request(const PagesArgs& a, int r) {
    Request q;
    q.src = a.src[r];
    q.keep = a.keep[r];
    q.len = held_len(a, r);
    q.refused = static_cast<uint32_t>(q.src) >= static_cast<uint32_t>(a.R) || q.keep < 0 || q.keep > held_len(a, q.src);
    if (q.refused) {
        q.src = r;
        q.keep = q.len;
    }
    return q;
}
__device__ __forceinline__ int pages_of(const PagesArgs& a, int len) {
    return static_cast<int>((static_cast<uint32_t>(len) + (1u << a.page_shift) - 1u) >> a.page_shift);
}
__device__ __forceinline__ bool in_pool(const PagesArgs& a, int p) { return static_cast<uint32_t>(p) < static_cast<uint32_t>(a.pool); }
__device__ __forceinline__ const int32_t* table_row(const PagesArgs& a, int r) { return a.table + static_cast<size_t>(r) * a.S; }

// --- words
__device__ __forceinline__ void clear_words(const PagesArgs& a, uint32_t* words, int id, int n) {
    for (int p = id; p < a.pool; p += n) words[p] = kNone;
}
// A wave's claims for parts of 256 entries of the requests' rows.
template <bool FORK>
__device__ __forceinline__ void claims(const PagesArgs& a, uint32_t* words, int wave, int waves, int lane) {
    const int parts = (a.S + 255) / 256;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += waves) {
        const int r = static_cast<int>(i / parts), j0 = static_cast<int>(i - static_cast<int64_t>(r) * parts) * 256;
        Request q{r, 0, 0, false};
        if constexpr (FORK) q = request(a, r);
        else q.len = held_len(a, r);
        const int held = pages_of(a, q.len), whole = q.keep >> a.page_shift;
        const bool part = FORK && (q.keep & ((1 << a.page_shift) - 1));
        const uint32_t key = 1u + (q.src == r ? r : a.R + r);
        const int32_t *own = table_row(a, r), *from = table_row(a, q.src);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 64 * e + lane;
            const bool kept = FORK && (j < whole || (j == whole && part));
            if (j < held && !(kept && q.src == r)) {  // (its own pages that it keeps are claimed as such)
                const int p = own[j];
                if (in_pool(a, p)) atomicMin(&words[p], kHeld);
            }
            if (kept) {
                const int p = from[j];
                if (in_pool(a, p)) atomicMin(&words[p], j < whole ? 0u : key);
            }
        }
    }
}

// --- sums over a workgroup of up to 1024 threads, in thread order: the value
// before this thread's, and the total.  s: 17 words of LDS.
__device__ __forceinline__ int block_before(int v, int& total, int32_t* s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (blockDim.x + 63) >> 6;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(x, o, 64);
        x += lane >= o ? t : 0;
    }
    __syncthreads();  // (the last call's reads are done)
    if (lane == 63) s[wave] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < waves; ++w) {
        before += w < wave ? s[w] : 0;
        total += s[w];
    }
    return before + x - v;
}

// The requests' outcomes, by one workgroup: lengths, fresh pages, the list of
// copies (its used places), copies and refusals in all (the same in every thread).
__device__ __forceinline__ void decide(const PagesArgs& a, const uint32_t* words, int32_t* s, int& copies, int& refusals) {
    int head = a.state[0] % a.pool;
    if (head < 0) head += a.pool;
    const int count = min(max(a.state[1], 0), a.pool);
    copies = refusals = 0;
    int asked = 0;
    for (int r0 = 0; r0 < a.R; r0 += blockDim.x) {
        const int r = r0 + threadIdx.x;
        Request q{0, 0, 0, false};
        int last = -1;
        bool copy = false;
        if (r < a.R) {
            q = request(a, r);
            if (q.keep & ((1 << a.page_shift) - 1)) {
                last = table_row(a, q.src)[q.keep >> a.page_shift];
                copy = in_pool(a, last) && words[last] != 1u + (q.src == r ? r : a.R + r);
            }
        }
        int total, all;
        const int at = asked + block_before(copy ? 1 : 0, total, s);
        const bool given = copy && at < count, cut = copy && !given;
        if (r < a.R) {
            a.o_len[r] = cut ? q.keep >> a.page_shift << a.page_shift : q.keep;
            int fresh = -1;
            if (given) {
                fresh = a.ring[(static_cast<uint32_t>(head) + static_cast<uint32_t>(at)) % static_cast<uint32_t>(a.pool)];
                a.o_frm[at] = last;
                a.o_to[at] = fresh;
            }
            a.fresh[r] = given ? fresh : -1;
        }
        block_before(cut || q.refused ? 1 : 0, all, s);
        asked += total;
        refusals += all;
    }
    copies = min(asked, count);
}

// Tables after a fork: a wave takes parts of 256 entries of the rows.
__device__ __forceinline__ void fork_tables(const PagesArgs& a, int wave, int waves, int lane) {
    const int parts = (a.S + 255) / 256;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += waves) {
        const int r = static_cast<int>(i / parts), j0 = static_cast<int>(i - static_cast<int64_t>(r) * parts) * 256;
        const Request q = request(a, r);
        const int now = a.o_len[r], n = pages_of(a, now), fresh = a.fresh[r];
        const int32_t* from = table_row(a, q.src);
        int32_t* to = a.table_out + static_cast<size_t>(r) * a.S;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 64 * e + lane;
            if (j < n) to[j] = j == n - 1 && fresh >= 0 ? fresh : from[j];
        }
    }
}

// Freed pages of [p0, p1) to the ring, `base` of them lying before.
__device__ __forceinline__ int fork_ring(const PagesArgs& a, const uint32_t* words, int p0, int p1, int base, int32_t* s) {
    int head = a.state[0] % a.pool;
    if (head < 0) head += a.pool;
    const int count = min(max(a.state[1], 0), a.pool);
    for (int c = p0; c < p1; c += blockDim.x) {
        const int p = c + threadIdx.x;
        const bool freed = p < p1 && words[p] == kHeld;
        int total;
        const int at = base + block_before(freed ? 1 : 0, total, s);
        if (freed && at < a.pool - count)
            a.ring[(static_cast<uint32_t>(head) + static_cast<uint32_t>(count) + static_cast<uint32_t>(at)) % static_cast<uint32_t>(a.pool)] = p;
        base += total;
    }
    return base;
}
__device__ __forceinline__ void fork_state(const PagesArgs& a, int copies, int refusals, int freed) {
    int head = a.state[0] % a.pool;
    if (head < 0) head += a.pool;
    const int count = min(max(a.state[1], 0), a.pool);
    a.o_state[0] = static_cast<int>((static_cast<uint32_t>(head) + static_cast<uint32_t>(copies)) % static_cast<uint32_t>(a.pool));
    a.o_state[1] = count - copies + min(freed, a.pool - count);
    a.o_state[2] = copies;
    a.o_state[3] = refusals;
}

// Pages of [p0, p1) of a pool being compacted, `base` held pages lying before
// and n in all.  With b held pages below it, a held page is the (n - 1 - b)-th
// from the top and a free page p the (p - b)-th from the bottom; the first K =
// (held pages at n or above) of each list change places (the first M of them,
// if the list is that short), and K = n less the held pages below n.
__device__ __forceinline__ int compact_lists(const PagesArgs& a, const uint32_t* words, int p0, int p1, int base, int n, int moves,
                                             int all, int32_t* s) {
    for (int c = p0; c < p1; c += blockDim.x) {
        const int p = c + threadIdx.x;
        const bool held = p < p1 && words[p] != kNone;
        int total;
        const int b = base + block_before(held ? 1 : 0, total, s);
        if (p < p1) {
            const int k = held ? n - 1 - b : p - b;
            const bool moved = k < moves;
            a.rank[p] = held && moved ? k : -1;
            if (moved) (held ? a.o_frm : a.o_to)[k] = p;
            if (held == moved) {  // free after the call: behind those free below it
                const int held_below = b + min(moves, p - b) - max(0, b - (n - moves));
                a.ring[p - held_below] = p;
            }
            if (held && k == moves && moves < all) a.o_state[3] = p + 1;  // the highest page that stays
        }
        base += total;
    }
    return base;
}
__device__ __forceinline__ void compact_tables(const PagesArgs& a, int wave, int waves, int lane) {
    const int parts = (a.S + 255) / 256;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += waves) {
        const int r = static_cast<int>(i / parts), j0 = static_cast<int>(i - static_cast<int64_t>(r) * parts) * 256;
        const int len = held_len(a, r), held = pages_of(a, len);
        if (j0 == 0 && lane == 0) a.o_len[r] = len;
        const int32_t* from = table_row(a, r);
        int32_t* to = a.table_out + static_cast<size_t>(r) * a.S;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 64 * e + lane;
            if (j >= held) continue;
            const int p = from[j], k = in_pool(a, p) ? a.rank[p] : -1;
            to[j] = k >= 0 ? a.o_to[k] : p;
        }
    }
}
__device__ __forceinline__ void compact_state(const PagesArgs& a, int n, int moves, int all) {
    a.o_state[0] = 0;
    a.o_state[1] = a.pool - n;
    a.o_state[2] = moves;
    if (moves == all) a.o_state[3] = n;
}
__device__ __forceinline__ void pad_lists(const PagesArgs& a, int used, int id, int n) {
    for (int i = used + id; i < a.M; i += n) a.o_frm[i] = a.o_to[i] = -1;
}
// Held pages below n, of a pool whose words these are (one workgroup).
__device__ __forceinline__ int count_words(const uint32_t* words, int p0, int p1, bool fork, int32_t* s) {
    int mine = 0, total;
    for (int p = p0 + threadIdx.x; p < p1; p += blockDim.x) mine += fork ? words[p] == kHeld : words[p] != kNone;
    block_before(mine, total, s);
    return total;
}

// ------------------------------------------------- one workgroup, words in LDS
template <bool FORK>
__global__ __launch_bounds__(1024) void pages_small_kernel(PagesArgs a) {
    extern __shared__ uint32_t s_words[];
    __shared__ int32_t s_scan[17];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6), waves = blockDim.x >> 6;
    clear_words(a, s_words, tid, blockDim.x);
    __syncthreads();
    claims<FORK>(a, s_words, wave, waves, lane);
    __syncthreads();
    if constexpr (FORK) {
        int copies, refusals;
        decide(a, s_words, s_scan, copies, refusals);
        __syncthreads();  // (o_len and fresh, read below, are written)
        fork_tables(a, wave, waves, lane);
        const int freed = fork_ring(a, s_words, 0, a.pool, 0, s_scan);
        if (tid == 0) fork_state(a, copies, refusals, freed);
        pad_lists(a, copies, tid, blockDim.x);
    } else {
        const int n = count_words(s_words, 0, a.pool, false, s_scan);
        const int all = n - count_words(s_words, 0, n, false, s_scan), moves = min(all, a.M);
        compact_lists(a, s_words, 0, a.pool, 0, n, moves, all, s_scan);
        __syncthreads();  // (ranks and places are written)
        compact_tables(a, wave, waves, lane);
        if (tid == 0) compact_state(a, n, moves, all);
        pad_lists(a, moves, tid, blockDim.x);
    }
}

// ------------------------------------------------------- a launch for each phase
__global__ __launch_bounds__(256) void pages_clear_kernel(PagesArgs a) {
    clear_words(a, a.words, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}
template <bool FORK>
__global__ __launch_bounds__(256) void pages_claim_kernel(PagesArgs a) {
    claims<FORK>(a, a.words, blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6), gridDim.x * 4, threadIdx.x & 63);
}
// Workgroup 0 of a fork decides; the others (all, for a compaction) sum a segment each.
template <bool FORK>
__global__ __launch_bounds__(1024) void pages_sum_kernel(PagesArgs a) {
    __shared__ int32_t s_scan[17];
    int seg = blockIdx.x;
    if constexpr (FORK) {
        if (seg == 0) {
            int copies, refusals;
            decide(a, a.words, s_scan, copies, refusals);
            if (threadIdx.x == 0) {
                a.o_state[2] = copies;
                a.o_state[3] = refusals;
            }
            return;
        }
        --seg;
    }
    const int p0 = seg * kSeg, total = count_words(a.words, p0, min(p0 + kSeg, a.pool), FORK, s_scan);
    if (threadIdx.x == 0) a.sums[seg] = total;
}
// Sum of the segments before seg, and of all (the same in every thread).
__device__ __forceinline__ int sums_before(const PagesArgs& a, int seg, int& all, int32_t* s) {
    const int segs = (a.pool + kSeg - 1) / kSeg;
    int before = 0, mine = 0, total;
    for (int i = threadIdx.x; i < segs; i += blockDim.x) {
        mine += a.sums[i];
        before += i < seg ? a.sums[i] : 0;
    }
    block_before(mine, all, s);
    block_before(before, total, s);
    return total;
}
__global__ __launch_bounds__(1024) void fork_write_kernel(PagesArgs a, int segs) {
    __shared__ int32_t s_scan[17];
    if (static_cast<int>(blockIdx.x) < segs) {
        const int seg = blockIdx.x, p0 = seg * kSeg;
        int all;
        const int base = sums_before(a, seg, all, s_scan);
        fork_ring(a, a.words, p0, min(p0 + kSeg, a.pool), base, s_scan);
        if (seg == 0) {
            const int copies = a.o_state[2], refusals = a.o_state[3];
            if (threadIdx.x == 0) fork_state(a, copies, refusals, all);
        }
        return;
    }
    const int id = blockIdx.x - segs, n = gridDim.x - segs;
    fork_tables(a, id * 16 + wave_uniform(threadIdx.x >> 6), n * 16, threadIdx.x & 63);
    pad_lists(a, a.o_state[2], id * 1024 + threadIdx.x, n * 1024);
}
__global__ __launch_bounds__(1024) void compact_lists_kernel(PagesArgs a) {
    __shared__ int32_t s_scan[17];
    const int seg = blockIdx.x, p0 = seg * kSeg;
    int n, all;
    const int base = sums_before(a, seg, n, s_scan);
    // held pages below n: whole segments from their sums, the one that n lies in counted
    const int at = n / kSeg, below = sums_before(a, at, all, s_scan);
    const int extra = n < a.pool ? count_words(a.words, at * kSeg, n, false, s_scan) : 0;
    const int want = n < a.pool ? n - below - extra : 0, moves = min(want, a.M);
    compact_lists(a, a.words, p0, min(p0 + kSeg, a.pool), base, n, moves, want, s_scan);
    if (seg == 0 && threadIdx.x == 0) compact_state(a, n, moves, want);
    pad_lists(a, moves, seg * 1024 + threadIdx.x, gridDim.x * 1024);
}
__global__ __launch_bounds__(256) void compact_tables_kernel(PagesArgs a) {
    compact_tables(a, blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6), gridDim.x * 4, threadIdx.x & 63);
}

static PagesArgs pages_args(const bitq_kv_pages_desc& d, void* result, void* ws) {
    const KvPagesLayout L = kv_pages_layout(d);
    PagesArgs a{};
    uint8_t *b = static_cast<uint8_t*>(result), *w = static_cast<uint8_t*>(ws);
    auto at = [](uint8_t* p, size_t off) { return reinterpret_cast<int32_t*>(p + off); };
    a.o_state = at(b, 0);
    a.o_len = at(b, L.off_len);
    a.o_frm = at(b, L.off_frm);
    a.o_to = at(b, L.off_to);
    a.words = reinterpret_cast<uint32_t*>(w);
    a.sums = at(w, L.off_sums);
    a.fresh = at(w, L.off_fresh);
    a.rank = at(w, L.off_rank);
    a.R = d.requests;
    a.S = d.table_stride;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(d.page));
    a.pool = d.pool;
    a.M = d.moves;
    return a;
}

template <bool FORK>
static int launch_pages(const bitq_kv_pages_desc& d, const PagesArgs& a, hipStream_t st) {
    const int64_t parts = static_cast<int64_t>(d.requests) * ((d.table_stride + 255) / 256);  // waves' work of a table
    if (kv_pages_small(d)) {
        const size_t lds = 4 * static_cast<size_t>(d.pool);
        if (lds > 48 * 1024) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(pages_small_kernel<FORK>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
            if (e != hipSuccess) return static_cast<int>(e);
        }
        hipLaunchKernelGGL((pages_small_kernel<FORK>), dim3(1), dim3(1024), lds, st, a);
        return static_cast<int>(hipGetLastError());
    }
    const unsigned segs = (d.pool + kSeg - 1) / kSeg;
    const unsigned table = static_cast<unsigned>(std::min<int64_t>(2048, (parts + 3) / 4));
    hipLaunchKernelGGL(pages_clear_kernel, dim3(std::min(1024u, (d.pool + 1023u) / 1024u)), dim3(256), 0, st, a);
    hipLaunchKernelGGL((pages_claim_kernel<FORK>), dim3(table), dim3(256), 0, st, a);
    hipLaunchKernelGGL((pages_sum_kernel<FORK>), dim3(segs + (FORK ? 1 : 0)), dim3(1024), 0, st, a);
    if constexpr (FORK) {
        hipLaunchKernelGGL(fork_write_kernel, dim3(segs + std::max(1u, (table + 3) / 4)), dim3(1024), 0, st, a, static_cast<int>(segs));
    } else {
        hipLaunchKernelGGL(compact_lists_kernel, dim3(segs), dim3(1024), 0, st, a);
        hipLaunchKernelGGL(compact_tables_kernel, dim3(table), dim3(256), 0, st, a);
    }
    return static_cast<int>(hipGetLastError());
}

int launch_kv_fork(const bitq_kv_pages_desc& d, const int32_t* src, const int32_t* keep, const int32_t* len, int32_t* ring,
                   const int32_t* state, const int32_t* table, int32_t* table_out, void* result, void* ws, void* stream) {
    PagesArgs a = pages_args(d, result, ws);
    a.src = src, a.keep = keep, a.len = len, a.ring = ring, a.state = state, a.table = table, a.table_out = table_out;
    return launch_pages<true>(d, a, static_cast<hipStream_t>(stream));
}

int launch_kv_compact(const bitq_kv_pages_desc& d, const int32_t* len, const int32_t* table, int32_t* table_out, int32_t* ring,
                      void* result, void* ws, void* stream) {
    PagesArgs a = pages_args(d, result, ws);
    a.len = len, a.ring = ring, a.table = table, a.table_out = table_out;
    return launch_pages<false>(d, a, static_cast<hipStream_t>(stream));
}

// ====================================================================== copies
// A page's keys lie in a row, and so do its values and scales: a workgroup
// takes 16 KB of one of these sections at a time, pairs outermost.  Bound by
// HBM (each byte read and written once).
struct CopyArgs {
    const int32_t *frm, *to;
    uint8_t* cache;
    size_t off_v, off_ks, off_vs;
    uint32_t kv_bytes, sc_bytes;  // of a page's keys (values), and of its scales of either
    int moves, pages, pieces, pieces_kv;
};
constexpr uint32_t kPiece = 256 * 16 * 4;

__global__ __launch_bounds__(256) void kv_copy_kernel(CopyArgs a) {
    const int64_t items = static_cast<int64_t>(a.moves) * a.pieces;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int m = static_cast<int>(i / a.pieces), piece = static_cast<int>(i - static_cast<int64_t>(m) * a.pieces);
        const int from = a.frm[m], to = a.to[m];
        if (static_cast<uint32_t>(from) >= static_cast<uint32_t>(a.pages) || static_cast<uint32_t>(to) >= static_cast<uint32_t>(a.pages) ||
            from == to)
            continue;
        // sections: keys, values, then both scales as one piece each
        uint8_t* base = a.cache;
        uint32_t size = a.kv_bytes, at = 0;
        if (piece < 2 * a.pieces_kv) {
            const bool v = piece >= a.pieces_kv;
            if (v) base += a.off_v;
            at = static_cast<uint32_t>(piece - (v ? a.pieces_kv : 0)) * kPiece;
        } else {
            const int rest = piece - 2 * a.pieces_kv, per = (a.pieces - 2 * a.pieces_kv) / 2;
            base += rest >= per ? a.off_vs : a.off_ks;
            size = a.sc_bytes;
            at = static_cast<uint32_t>(rest % per) * kPiece;
        }
        const uint8_t* x = base + static_cast<size_t>(from) * size;
        uint8_t* y = base + static_cast<size_t>(to) * size;
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t o = at + (e * 256 + threadIdx.x) * 16;
            if (o < size) v[e] = *reinterpret_cast<const uint4*>(x + o);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t o = at + (e * 256 + threadIdx.x) * 16;
            if (o < size) *reinterpret_cast<uint4*>(y + o) = v[e];
        }
    }
}

int launch_kv_copy(const bitq_kvdesc& kv, const int32_t* frm, const int32_t* to, int moves, void* cache, void* stream) {
    const KvLayout L = kv_layout(kv);
    CopyArgs a{};
    a.frm = frm;
    a.to = to;
    a.cache = static_cast<uint8_t*>(cache);
    a.off_v = L.off_v;
    a.off_ks = L.off_ks;
    a.off_vs = L.off_vs;
    // (a page has 8 tokens or more: every section is a multiple of 32 bytes)
    const uint32_t rows = static_cast<uint32_t>(kv.page) * kv.kv_heads;  // (<= 2^20)
    a.kv_bytes = rows * L.Dp * (kv.dtype == BITQ_KV_BF16 ? 2 : 1);
    a.sc_bytes = rows * 4;
    a.moves = moves;
    a.pages = kv.pages;
    a.pieces_kv = (a.kv_bytes + kPiece - 1) / kPiece;
    a.pieces = 2 * a.pieces_kv + (kv.dtype == BITQ_KV_INT8 ? 2 * static_cast<int>((a.sc_bytes + kPiece - 1) / kPiece) : 0);
    const int64_t items = static_cast<int64_t>(moves) * a.pieces;
    hipLaunchKernelGGL(kv_copy_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, 256 * 16))), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
