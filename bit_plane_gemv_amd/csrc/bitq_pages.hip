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
//
// Bound by latency: a fork of 64 requests of up to 64 pages 10.4 us in one
// launch, of 256 requests of up to 128 pages 14.6 us in four; a compaction of 257
// pages 5.5 us in one, of 16385 pages 26 us in five (both sides of the rule:
// kv_pages_small).
constexpr uint32_t kNone = 0xFFFFFFFFu, kHeld = 0xFFFFFFFEu;

struct PagesArgs {
    const int32_t *src, *keep, *len, *table, *state;
    int32_t *ring, *table_out;
    int32_t *o_state, *o_len, *o_frm, *o_to;
    uint32_t* words;   // [pool]
    int32_t* sums;     // [segments]: freed (fork) or held (compact) pages of each
    int32_t* fresh;    // fork: [R] the copy's page (-1: none)
    int32_t* rank;     // compact: [pool] a moved page's place in the list (else -1)
    struct Request* reqs;  // [R]
    int R, S, page_shift, pool, M;
    int seg;           // pages of the pool that a workgroup sums
};

// A request as taken (its own tokens, if what it asks for is refused), by the
// first phase, so that the next ones wait for no chain of loads.
struct __align__(16) Request {
    int src, keep, len, refused;
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
template <bool FORK>
__device__ __forceinline__ void resolve(const PagesArgs& a, Request* reqs, int id, int n) {
    for (int r = id; r < a.R; r += n) {
        Request q{r, 0, 0, 0};
        if constexpr (FORK) q = request(a, r);
        else q.len = held_len(a, r);
        reqs[r] = q;
    }
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
// A wave's claims for parts of 64 entries of the requests' rows, kParts of them
// at a time (their loads are on their way together).
constexpr int kParts = 4;
template <bool FORK>
__device__ __forceinline__ void claims(const PagesArgs& a, const Request* reqs, uint32_t* words, int wave, int waves, int lane) {
    const uint32_t parts = (a.S + 63) / 64;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += static_cast<int64_t>(waves) * kParts) {
        int p_own[kParts], p_from[kParts];
        uint32_t claim[kParts];
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
            const int64_t item = i + static_cast<int64_t>(u) * waves;
            p_own[u] = p_from[u] = -1;
            claim[u] = kHeld;
            if (item >= items) continue;
            const int r = items <= UINT32_MAX ? static_cast<uint32_t>(item) / parts : static_cast<int>(item / parts);
            const int j = static_cast<int>(item - static_cast<int64_t>(r) * parts) * 64 + lane;
            const Request q = reqs[r];
            const int whole = q.keep >> a.page_shift;
            const bool part = FORK && (q.keep & ((1 << a.page_shift) - 1));
            const bool kept = FORK && (j < whole || (j == whole && part));
            claim[u] = j < whole ? 0u : 1u + (q.src == r ? r : a.R + r);
            if (j < pages_of(a, q.len) && !(kept && q.src == r)) p_own[u] = table_row(a, r)[j];  // (its own pages that it keeps are claimed as such)
            if (kept) p_from[u] = table_row(a, q.src)[j];
        }
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
            if (in_pool(a, p_own[u])) atomicMin(&words[p_own[u]], kHeld);
            if (FORK && in_pool(a, p_from[u])) atomicMin(&words[p_from[u]], claim[u]);
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
__device__ __forceinline__ void decide(const PagesArgs& a, const Request* reqs, const uint32_t* words, int32_t* s, int& copies,
                                       int& refusals) {
    int head = a.state[0] % a.pool;
    if (head < 0) head += a.pool;
    const int count = min(max(a.state[1], 0), a.pool);
    copies = refusals = 0;
    int asked = 0;
    for (int r0 = 0; r0 < a.R; r0 += blockDim.x) {
        const int r = r0 + threadIdx.x;
        Request q{0, 0, 0, 0};
        int last = -1;
        bool copy = false;
        if (r < a.R) {
            q = reqs[r];
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

// Tables after a fork: a wave takes parts of 64 entries of the rows, as in claims().
__device__ __forceinline__ void fork_tables(const PagesArgs& a, const Request* reqs, int wave, int waves, int lane) {
    const uint32_t parts = (a.S + 63) / 64;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += static_cast<int64_t>(waves) * kParts) {
        int p[kParts];
        int32_t* to[kParts];
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
            const int64_t item = i + static_cast<int64_t>(u) * waves;
            to[u] = nullptr;
            p[u] = 0;
            if (item >= items) continue;
            const int r = items <= UINT32_MAX ? static_cast<uint32_t>(item) / parts : static_cast<int>(item / parts);
            const int j = static_cast<int>(item - static_cast<int64_t>(r) * parts) * 64 + lane;
            const int n = pages_of(a, a.o_len[r]), fresh = a.fresh[r];
            if (j < n) {
                to[u] = a.table_out + static_cast<size_t>(r) * a.S + j;
                p[u] = table_row(a, reqs[r].src)[j];
                if (j == n - 1 && fresh >= 0) p[u] = fresh;
            }
        }
#pragma unroll
        for (int u = 0; u < kParts; ++u)
            if (to[u]) *to[u] = p[u];
    }
}

// The words of pages p .. p + PER - 1 (kNone from p1 on).
template <int PER>
__device__ __forceinline__ void words_of(const uint32_t* words, int p, int p1, uint32_t (&w)[PER]) {
#pragma unroll
    for (int e = 0; e < PER; ++e) w[e] = p + e < p1 ? words[p + e] : kNone;
}

// PER: pages of a thread, next to each other.  1 keeps the stores of a wave in a
// row (segments of a pool in the workspace: 18 -> 6 us with 16385 pages against
// 8); 8 saves rounds of the sum (one workgroup, 4165 pages: 13.8 -> 10.6 us); a
// compaction stores more: 4 (4565 pages: 13.5 us, 1 14.3, 8 15.1).
// Freed pages of [p0, p1) to the ring, `base` of them lying before.
template <int PER>
__device__ __forceinline__ int fork_ring(const PagesArgs& a, const uint32_t* words, int p0, int p1, int base, int32_t* s) {
    int head = a.state[0] % a.pool;
    if (head < 0) head += a.pool;
    const int count = min(max(a.state[1], 0), a.pool);
    for (int c = p0; c < p1; c += PER * blockDim.x) {
        const int p = c + PER * threadIdx.x;
        uint32_t w[PER];
        words_of(words, p, p1, w);
        int mine = 0, total;
#pragma unroll
        for (int e = 0; e < PER; ++e) mine += w[e] == kHeld;
        int at = base + block_before(mine, total, s);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (w[e] != kHeld) continue;
            if (at < a.pool - count)
                a.ring[(static_cast<uint32_t>(head) + static_cast<uint32_t>(count) + static_cast<uint32_t>(at)) % static_cast<uint32_t>(a.pool)] = p + e;
            ++at;
        }
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
template <int PER>
__device__ __forceinline__ int compact_lists(const PagesArgs& a, const uint32_t* words, int p0, int p1, int base, int n, int moves,
                                             int all, int32_t* s) {
    for (int c = p0; c < p1; c += PER * blockDim.x) {
        const int q = c + PER * threadIdx.x;
        uint32_t w[PER];
        words_of(words, q, p1, w);
        int mine = 0, total;
#pragma unroll
        for (int e = 0; e < PER; ++e) mine += w[e] != kNone;
        int b = base + block_before(mine, total, s);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int p = q + e;
            const bool held = w[e] != kNone;
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
            b += held;
        }
        base += total;
    }
    return base;
}
__device__ __forceinline__ void compact_tables(const PagesArgs& a, const Request* reqs, int wave, int waves, int lane) {
    const uint32_t parts = (a.S + 63) / 64;
    const int64_t items = static_cast<int64_t>(a.R) * parts;
    for (int64_t i = wave; i < items; i += static_cast<int64_t>(waves) * kParts) {
        int p[kParts], k[kParts];
        int32_t* to[kParts];
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
            const int64_t item = i + static_cast<int64_t>(u) * waves;
            to[u] = nullptr;
            p[u] = -1;
            if (item >= items) continue;
            const int r = items <= UINT32_MAX ? static_cast<uint32_t>(item) / parts : static_cast<int>(item / parts);
            const int j = static_cast<int>(item - static_cast<int64_t>(r) * parts) * 64 + lane;
            const int len = reqs[r].len;
            if (j == 0) a.o_len[r] = len;
            if (j < pages_of(a, len)) {
                to[u] = a.table_out + static_cast<size_t>(r) * a.S + j;
                p[u] = table_row(a, r)[j];
            }
        }
#pragma unroll
        for (int u = 0; u < kParts; ++u) k[u] = in_pool(a, p[u]) ? a.rank[p[u]] : -1;
#pragma unroll
        for (int u = 0; u < kParts; ++u)
            if (to[u]) *to[u] = k[u] >= 0 ? a.o_to[k[u]] : p[u];
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
    extern __shared__ __align__(16) uint8_t s_mem[];
    __shared__ int32_t s_scan[17];
    Request* reqs = reinterpret_cast<Request*>(s_mem);
    uint32_t* words = reinterpret_cast<uint32_t*>(s_mem + a.R * sizeof(Request));
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6), waves = blockDim.x >> 6;
    resolve<FORK>(a, reqs, tid, blockDim.x);
    clear_words(a, words, tid, blockDim.x);
    __syncthreads();
    claims<FORK>(a, reqs, words, wave, waves, lane);
    __syncthreads();
    if constexpr (FORK) {
        int copies, refusals;
        decide(a, reqs, words, s_scan, copies, refusals);
        __syncthreads();  // (o_len and fresh, read below, are written)
        fork_tables(a, reqs, wave, waves, lane);
        const int freed = a.pool > 1024 ? fork_ring<8>(a, words, 0, a.pool, 0, s_scan) : fork_ring<1>(a, words, 0, a.pool, 0, s_scan);
        if (tid == 0) fork_state(a, copies, refusals, freed);
        pad_lists(a, copies, tid, blockDim.x);
    } else {
        const int n = count_words(words, 0, a.pool, false, s_scan);
        const int all = n - count_words(words, 0, n, false, s_scan), moves = min(all, a.M);
        if (a.pool > 2048) compact_lists<4>(a, words, 0, a.pool, 0, n, moves, all, s_scan);
        else compact_lists<1>(a, words, 0, a.pool, 0, n, moves, all, s_scan);
        __syncthreads();  // (ranks and places are written)
        compact_tables(a, reqs, wave, waves, lane);
        if (tid == 0) compact_state(a, n, moves, all);
        pad_lists(a, moves, tid, blockDim.x);
    }
}

// ------------------------------------------------------- a launch for each phase
template <bool FORK>
__global__ __launch_bounds__(256) void pages_clear_kernel(PagesArgs a) {
    resolve<FORK>(a, a.reqs, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
    clear_words(a, a.words, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}
template <bool FORK>
__global__ __launch_bounds__(256) void pages_claim_kernel(PagesArgs a) {
    claims<FORK>(a, a.reqs, a.words, blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6), gridDim.x * 4, threadIdx.x & 63);
}
// Workgroup 0 of a fork decides; the others (all, for a compaction) sum a segment each.
template <bool FORK>
__global__ __launch_bounds__(1024) void pages_sum_kernel(PagesArgs a) {
    __shared__ int32_t s_scan[17];
    int seg = blockIdx.x;
    if constexpr (FORK) {
        if (seg == 0) {
            int copies, refusals;
            decide(a, a.reqs, a.words, s_scan, copies, refusals);
            if (threadIdx.x == 0) {
                a.o_state[2] = copies;
                a.o_state[3] = refusals;
            }
            return;
        }
        --seg;
    }
    const int p0 = seg * a.seg, total = count_words(a.words, p0, min(p0 + a.seg, a.pool), FORK, s_scan);
    if (threadIdx.x == 0) a.sums[seg] = total;
}
// Sum of the segments before seg, and of all (the same in every thread).
__device__ __forceinline__ int sums_before(const PagesArgs& a, int seg, int& all, int32_t* s) {
    const int segs = (a.pool + a.seg - 1) / a.seg;
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
        const int seg = blockIdx.x, p0 = seg * a.seg;
        int all;
        const int base = sums_before(a, seg, all, s_scan);
        fork_ring<1>(a, a.words, p0, min(p0 + a.seg, a.pool), base, s_scan);
        if (seg == 0) {
            const int copies = a.o_state[2], refusals = a.o_state[3];
            if (threadIdx.x == 0) fork_state(a, copies, refusals, all);
        }
        return;
    }
    const int id = blockIdx.x - segs, n = gridDim.x - segs;
    fork_tables(a, a.reqs, id * 16 + wave_uniform(threadIdx.x >> 6), n * 16, threadIdx.x & 63);
    pad_lists(a, a.o_state[2], id * 1024 + threadIdx.x, n * 1024);
}
__global__ __launch_bounds__(1024) void compact_lists_kernel(PagesArgs a) {
    __shared__ int32_t s_scan[17];
    const int seg = blockIdx.x, p0 = seg * a.seg;
    int n, all;
    const int base = sums_before(a, seg, n, s_scan);
    // held pages below n: whole segments from their sums, the one that n lies in counted
    const int at = n / a.seg, below = sums_before(a, at, all, s_scan);
    const int extra = n < a.pool ? count_words(a.words, at * a.seg, n, false, s_scan) : 0;
    const int want = n < a.pool ? n - below - extra : 0, moves = min(want, a.M);
    compact_lists<1>(a, a.words, p0, min(p0 + a.seg, a.pool), base, n, moves, want, s_scan);
    if (seg == 0 && threadIdx.x == 0) compact_state(a, n, moves, want);
    pad_lists(a, moves, seg * 1024 + threadIdx.x, gridDim.x * 1024);
}
__global__ __launch_bounds__(256) void compact_tables_kernel(PagesArgs a) {
    compact_tables(a, a.reqs, blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6), gridDim.x * 4, threadIdx.x & 63);
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
    a.reqs = reinterpret_cast<Request*>(w + L.off_reqs);
    a.R = d.requests;
    a.S = d.table_stride;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(d.page));
    a.pool = d.pool;
    a.M = d.moves;
    a.seg = kv_pages_segment(d);
    return a;
}

template <bool FORK>
static int launch_pages(const bitq_kv_pages_desc& d, const PagesArgs& a, hipStream_t st) {
    const int64_t parts = static_cast<int64_t>(d.requests) * ((d.table_stride + 63) / 64);  // waves' work of a table
    if (kv_pages_small(d)) {
        const size_t lds = 4 * static_cast<size_t>(d.pool) + sizeof(Request) * static_cast<size_t>(d.requests);
        if (lds > 48 * 1024) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(pages_small_kernel<FORK>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
            if (e != hipSuccess) return static_cast<int>(e);
        }
        hipLaunchKernelGGL((pages_small_kernel<FORK>), dim3(1), dim3(1024), lds, st, a);
        return static_cast<int>(hipGetLastError());
    }
    const unsigned segs = (d.pool + a.seg - 1) / a.seg;
    const unsigned table = static_cast<unsigned>(std::min<int64_t>(2048, (parts + 3) / 4));
    const unsigned clear = static_cast<unsigned>(std::min(1024, (std::max(d.pool, d.requests) + 255) / 256));
    hipLaunchKernelGGL((pages_clear_kernel<FORK>), dim3(clear), dim3(256), 0, st, a);
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
// takes 16 KB of one of these sections, blockIdx.x of a page's pieces, of the
// pages blockIdx.y, blockIdx.y + gridDim.y, ...  Bound by HBM (each byte read and
// written once): 3700 pages of 64 KB 90 us, 5.4 TB/s; 48 pages 2.6 us.  No
// element of a lane's registers is written under a condition: such arrays were
// moved to LDS by the compiler, which then reads the workgroup's size from the
// dispatch packet in host memory (15 us whatever was copied).
struct CopyArgs {
    const int32_t *frm, *to;
    uint8_t* cache;
    size_t off_v, off_ks, off_vs;
    uint32_t kv_bytes, sc_bytes;  // of a page's keys (values), and of its scales of either
    int moves, pages, pieces_kv, pieces_sc;
};
constexpr uint32_t kPiece = 256 * 16 * 4;
constexpr int kCopyGroups = 8192;

__global__ __launch_bounds__(256) void kv_copy_kernel(CopyArgs a) {
    // sections: keys, values, then the scales of both
    int piece = blockIdx.x;
    uint8_t* base = a.cache;
    uint32_t size = a.kv_bytes;
    if (piece >= 2 * a.pieces_kv) {
        piece -= 2 * a.pieces_kv;
        base += piece >= a.pieces_sc ? a.off_vs : a.off_ks;
        if (piece >= a.pieces_sc) piece -= a.pieces_sc;
        size = a.sc_bytes;
    } else if (piece >= a.pieces_kv) {
        piece -= a.pieces_kv;
        base += a.off_v;
    }
    // (a place past the section's end is its last one: its lanes copy the same bytes)
    uint32_t at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = min(static_cast<uint32_t>(piece) * kPiece + (e * 256 + threadIdx.x) * 16, size - 16);
    for (int m = blockIdx.y; m < a.moves; m += gridDim.y) {
        const int from = a.frm[m], to = a.to[m];
        if (static_cast<uint32_t>(from) >= static_cast<uint32_t>(a.pages) || static_cast<uint32_t>(to) >= static_cast<uint32_t>(a.pages) ||
            from == to)
            continue;
        const uint8_t* x = base + static_cast<size_t>(from) * size;
        uint8_t* y = base + static_cast<size_t>(to) * size;
        const uint4 v0 = *reinterpret_cast<const uint4*>(x + at[0]), v1 = *reinterpret_cast<const uint4*>(x + at[1]);
        const uint4 v2 = *reinterpret_cast<const uint4*>(x + at[2]), v3 = *reinterpret_cast<const uint4*>(x + at[3]);
        *reinterpret_cast<uint4*>(y + at[0]) = v0;
        *reinterpret_cast<uint4*>(y + at[1]) = v1;
        *reinterpret_cast<uint4*>(y + at[2]) = v2;
        *reinterpret_cast<uint4*>(y + at[3]) = v3;
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
    a.pieces_sc = kv.dtype == BITQ_KV_INT8 ? (a.sc_bytes + kPiece - 1) / kPiece : 0;
    const int pieces = 2 * (a.pieces_kv + a.pieces_sc);  // (<= 2^16 + 2^9)
    const int rows_y = std::min(moves, std::max(1, std::min(65535, kCopyGroups / pieces)));
    hipLaunchKernelGGL(kv_copy_kernel, dim3(pieces, rows_y), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return static_cast<int>(hipGetLastError());
}

}  // namespace bitq
