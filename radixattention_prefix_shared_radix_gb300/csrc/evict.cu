// Tokens leave a cache by their scores: for each request the pages that stay
// are found, and its rows of slots, scores and positions close up.
//
// A row's pages of P positions [0, n): those before `head` (sinks) and from
// `first` on (recent ones, and a last page that is not full) stay; of the
// others, whose score is their highest token's, the `more` highest stay, the
// earlier of equal ones.  Which score is the lowest that stays is found digit
// by digit (radix selection): scores become whole numbers of the same order,
// and four rounds each count the 256 values of the next eight bits among the
// pages that agree with the digits found so far.
//
// Work: a CTA per request, or a cluster of up to 16.  Its share of the row is read
// once, before the selection, and waits in registers for its places; the scores
// as whole numbers lie in shared memory.  A round counts into eight copies of its
// 256 counters (scores crowd a few exponents, and lanes of a warp that meet in one
// counter take turns); one warp finds the digit; a cluster's CTAs first read each
// other's counts through distributed shared memory.  Kept pages are numbered in
// order, eight a thread, with one exchange of the CTAs' totals, and every value
// goes to its place.  Places only get smaller and every read comes before the
// exchange, so a row may be moved onto itself.
// What bounds it is a chain of dependent steps, not bytes.  Calls that keep all
// (launch, reads, stores in order), then what calls that keep only what must stay
// take more (numbers, stores in other places), then the rounds: 64 rows of 2048
// cut to a quarter 2.3 + 1.9 + 2.8 us, 64 of 8192 3.5 + 3.6 + 4.8, 4 of 100000 to
// 131072 in pages of 16 3.5 + 6.7 + 9.2 (barriers of 16 CTAs in both), 4 of 500000
// 12 + 29 + 12 (places looked up in other CTAs' shares, a barrier for every 65536
// positions); the bytes' times at the copy's rate: 0.3, 1.3, 1.3, 5.  Rounds that
// went through one set of counters, read by every warp with bank conflicts, took
// 1.7 us each; rows read again for the moves, and places looked up across the
// cluster, cost another 2 to 4.
// The launch goes by the tables' width, as the host does not see the lengths: 48
// rows of 100 to 2000 tokens take 6.5 us in tables of their width and 76 in tables
// of 131072 (48 clusters of 16 CTAs, an SM each); scores of 2048 over such a table
// 6.5 again.
//
// ["SGLang 深度拆解" §2.3: the cache keeps what its budget allows]

#include <cooperative_groups.h>

#include <algorithm>

#include "common.h"
#include "device_common.cuh"

namespace {

using namespace sgldev;
namespace cg = cooperative_groups;

constexpr int kMaxCluster = 16;         // (more than 8 need the opt-in)
constexpr int kEach = 8;                 // positions of a thread, where its CTA takes its share at once
constexpr int kMaxShare = 49152;         // pages of a CTA's share (shared memory)
constexpr int kCopies = 8, kCopyStride = 257;

struct EvictArgs {
    const float* scores;
    const int32_t *table, *positions, *lens, *budgets;
    float* scores_out;
    int32_t *table_out, *positions_out, *lens_out, *evicted, *count;
    int64_t scores_ld, ld, evicted_ld;
    uint32_t* err;
    int page, lg_page;                   // lg_page < 0: not a power of two
    int lanes;                           // lanes of a warp that share a page, where it is a power of two; else 1
    int sinks, recent;
    int lim;                             // positions of a row: the shorter of ld and scores_ld
    bool in_place;                       // some output is its input
};

// A score as a whole number of the same order; NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = x == x ? __float_as_uint(x + 0.f) : 0xff800000u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A CTA's share is at most kEach positions a thread: they are read once, at the
// start, and wait in registers for their places.
template <int T>
__global__ void __launch_bounds__(T, 1) evict_kernel(const __grid_constant__ EvictArgs a) {
    constexpr int kWarps = T / 32;
    static_assert(T >= 256 && T % 256 == 0 && kWarps <= 32, "a thread per digit, a lane per warp");
    extern __shared__ __align__(16) uint32_t share[];      // a page's score; then its place, or ~(kept pages before it) if it leaves
    __shared__ uint32_t hist[kCopies * kCopyStride];       // counts of the digits, a copy for every eighth lane
    __shared__ uint32_t counts[2][256];                    // this CTA's, from digit 255 down
    __shared__ __align__(16) uint32_t total[256];          // the cluster's
    __shared__ uint3 choice;                               // a digit, pages above it, pages at it
    __shared__ uint2 warp_counts[kWarps], cta_counts;      // (pages that surely stay, pages at the lowest kept score)
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), c = (int)cl.block_rank();
    const int r = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kCopies * kCopyStride; i += T) hist[i] = 0;
    grid_dep_wait();
    grid_dep_launch();
    int n = a.lens[r];                       // (lens_out may be lens)
    const int budget = max(__ldg(a.budgets + r), 0);
    if (n < 0 || n > a.lim) {
        if (c == 0 && tid == 0) atomicOr(a.err, 2u);
        n = max(0, min(n, a.lim));
    }
    const int P = a.page;
    auto page_of = [&](int p) { return a.lg_page >= 0 ? p >> a.lg_page : p / P; };
    const int pages = n > 0 ? page_of(n - 1) + 1 : 0;
    const int S = (pages + C - 1) / C;                     // pages of a share
    const int p0 = min(c * S, pages), np = min(S, pages - p0);       // this CTA's
    const int t0 = p0 * P, nt = min(n - t0, np * P);

    const float* const scores = a.scores + (int64_t)r * a.scores_ld + t0;
    const int32_t* const table = a.table + (int64_t)r * a.ld + t0;
    const int32_t* const positions = a.positions ? a.positions + (int64_t)r * a.ld + t0 : nullptr;
    float x[kEach];
    int slot[kEach], at[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int t = tid + e * T;
        if (t < nt) x[e] = scores[t];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int t = tid + e * T;
        if (t < nt) {
            slot[e] = table[t];
            if (positions) at[e] = positions[t];
        }
    }
    const int first = page_of(max(n - a.recent, 0));       // (recent 0: a last page that is not full stays)
    const int head = min(page_of(a.sinks) + (a.sinks - page_of(a.sinks) * P > 0), first);
    const int fixed = head * P + (n - first * P);
    const int more = min(max(page_of(max(budget - fixed, 0)), 0), first - head);
    const bool some = n > budget && more < first - head;   // some pages leave
    if (some) {
        if (P > 1) {
            for (int i = tid; i < np; i += T) share[i] = 0;
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int t = tid + e * T;
            uint32_t y = t < nt ? order_of(x[e]) : 0;
            if (P == 1) {
                if (t < nt) share[t] = y;
                continue;
            }
            // (pages start at multiples of P from t = 0 on: lanes of one page, side by side, agree first)
            bool one = true;
            for (int o = 1; o < a.lanes; o <<= 1) {
                y = max(y, __shfl_xor_sync(0xffffffffu, y, o));
                one = (lane & (2 * o - 1)) == 0;
            }
            if (one && t < nt) atomicMax(&share[page_of(t)], y);
        }
        __syncthreads();
        // lowest score that stays, and how many of those at it
        uint32_t low = 0xffffffffu, mask = 0, found = 0;
        int need = 0;
        if (more > 0) {
            const int m0 = max(head - p0, 0), m1 = min(first - p0, np);
            uint32_t key[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid + e * T;
                key[e] = i >= m0 && i < m1 ? share[i] : 0;           // (no score is 0)
            }
            int k = more;
#pragma unroll 1
            for (int pass = 0; pass < 4; ++pass) {
                const int shift = 24 - 8 * pass;
                uint32_t* const mine = hist + (lane & (kCopies - 1)) * kCopyStride;
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (key[e] && (key[e] & mask) == found) atomicAdd(mine + ((key[e] >> shift) & 255u), 1u);
                __syncthreads();
                if (tid < 256) {
                    uint32_t v = 0;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        v += hist[i * kCopyStride + 255 - tid];
                        hist[i * kCopyStride + 255 - tid] = 0;
                    }
                    (C > 1 ? counts[pass & 1] : total)[tid] = v;
                }
                if (C > 1) {
                    cl.sync();
                    if (tid < 256) {
                        uint32_t v = 0;
#pragma unroll
                        for (int b = 0; b < kMaxCluster; ++b)
                            if (b < C) v += cl.map_shared_rank(counts[pass & 1], b)[tid];
                        total[tid] = v;
                    }
                }
                __syncthreads();
                // the digit with fewer than k pages above it and at least k from it on:
                // lane l has digits 255 - 8 l .. 248 - 8 l
                if (warp == 0) {
                    const uint4 u0 = reinterpret_cast<const uint4*>(total)[2 * lane], u1 = reinterpret_cast<const uint4*>(total)[2 * lane + 1];
                    const uint32_t v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                    const uint32_t sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
                    uint32_t upto = sum;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += y;
                    }
                    uint32_t before = upto - sum;
                    if (before < (uint32_t)k && upto >= (uint32_t)k) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (before < (uint32_t)k && before + v[i] >= (uint32_t)k) choice = make_uint3(255 - 8 * lane - i, before, v[i]);
                            before += v[i];
                        }
                    }
                }
                __syncthreads();
                const uint32_t digit = choice.x, above = choice.y, size = choice.z;
                k -= (int)above;
                found |= digit << shift;
                mask |= 255u << shift;
                low = found;
                need = k;
                if (size == (uint32_t)k && found > 0) {    // all of these stay: no further digit matters
                    low = found - 1;
                    need = 0;
                    break;
                }
            }
        }
        // number the kept pages: a thread takes eight neighbouring ones
        uint32_t sure = 0, equal = 0;                      // of them, a bit each
        const int i0 = 8 * tid;
        if (i0 < np) {
            const uint4 u0 = *reinterpret_cast<const uint4*>(share + i0), u1 = *reinterpret_cast<const uint4*>(share + i0 + 4);
            const uint32_t v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = p0 + i0 + i;
                if (i0 + i >= np) continue;
                if (p < head || p >= first || v[i] > low)
                    sure |= 1u << i;
                else if (v[i] == low)
                    equal |= 1u << i;
            }
        }
        uint2 w = make_uint2(__popc(sure), __popc(equal));
        const uint2 own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, w.x, o), z = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) {
                w.x += y;
                w.y += z;
            }
        }
        if (lane == 31) warp_counts[warp] = w;
        __syncthreads();
        uint2 before = lane < kWarps ? warp_counts[lane] : make_uint2(0, 0);
        uint2 all = before;
        if (lane >= warp) before = make_uint2(0, 0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before.x += __shfl_xor_sync(0xffffffffu, before.x, o);
            before.y += __shfl_xor_sync(0xffffffffu, before.y, o);
        }
        if (C > 1) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                all.x += __shfl_xor_sync(0xffffffffu, all.x, o);
                all.y += __shfl_xor_sync(0xffffffffu, all.y, o);
            }
            if (tid == 0) cta_counts = all;
            cl.sync();
            uint2 o = lane < c ? *cl.map_shared_rank(&cta_counts, lane) : make_uint2(0, 0);
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, i);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, i);
            }
            before.x += o.x;
            before.y += o.y;
            cl.barrier_arrive();         // (this CTA's counts may be read until all have arrived: waited for at the end)
        }
        if (i0 < np) {
            uint32_t surely = before.x + w.x - own.x, equals = before.y + w.y - own.y, y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t place = surely + min(equals, (uint32_t)need);
                const bool s = sure >> i & 1u, q = equal >> i & 1u;
                y[i] = s || (q && equals < (uint32_t)need) ? place : ~place;
                surely += s;
                equals += q;
            }
            *reinterpret_cast<uint4*>(share + i0) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(share + i0 + 4) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        __syncthreads();
    }
    const int left = some ? n - (first - head - more) * P : n;
    if (c == 0 && tid == 0) {
        a.lens_out[r] = left;
        if (a.count) a.count[r] = n - left;
        if (a.evicted && n - left > a.evicted_ld) atomicOr(a.err, 2u);
    }
    float* const scores_out = a.scores_out + (int64_t)r * a.scores_ld;
    int32_t* const table_out = a.table_out + (int64_t)r * a.ld;
    int32_t* const positions_out = positions ? a.positions_out + (int64_t)r * a.ld : nullptr;
    // (in place, others' reads are done: every CTA read its share before the
    // barriers that came with the numbers)
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int t = tid + e * T;
        if (t >= nt) continue;
        int to = t0 + t;
        if (some) {
            const int page = page_of(t), rest = t - page * P, place = (int)share[page];
            // (a page that leaves: its place among those)
            if (place >= 0)
                to = place * P + rest;
            else
                to = ~((p0 + page - ~place) * P + rest);
        }
        if (to >= 0) {
            scores_out[to] = x[e];
            table_out[to] = slot[e];
            if (positions) positions_out[to] = at[e];
        } else if (a.evicted && ~to < a.evicted_ld) {
            a.evicted[(int64_t)r * a.evicted_ld + ~to] = slot[e];
        }
        if (t0 + t >= left) {
            scores_out[t0 + t] = 0.f;
            table_out[t0 + t] = -1;
            if (positions) positions_out[t0 + t] = -1;
        }
    }
    if (C > 1 && some) cl.barrier_wait();
}

// Longer rows: the row is moved front to back in rounds of the whole cluster,
// whose CTAs look places up in each other's shares.
__global__ void __launch_bounds__(1024, 1) evict_long_kernel(const __grid_constant__ EvictArgs a) {
    constexpr int kThreads = 1024, kWarps = kThreads / 32, kEach = 4;      // (positions of a thread per round of moves)
    static_assert(kThreads >= 256 && kWarps == 32, "a thread per digit, a lane per warp");
    extern __shared__ __align__(16) uint32_t share[];      // a page's score; then its place, or ~(kept pages before it) if it leaves
    __shared__ uint32_t hist[kCopies * kCopyStride];       // counts of the digits, a copy for every eighth lane
    __shared__ uint32_t counts[2][256], warp_sums[8];      // this CTA's, from digit 255 down
    __shared__ uint3 choice;                               // the digit, pages above it, pages at it
    __shared__ uint2 warp_counts[kWarps], cta_counts;      // (pages that surely stay, pages at the lowest kept score)
    cg::cluster_group cl = cg::this_cluster();
    constexpr int C = kMaxCluster;                         // (fewer CTAs: evict_kernel)
    const int c = (int)cl.block_rank();
    const int r = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    grid_dep_launch();
    int n = a.lens[r];                       // (lens_out may be lens)
    const int budget = max(__ldg(a.budgets + r), 0);
    if (n < 0 || n > a.lim) {
        if (c == 0 && tid == 0) atomicOr(a.err, 2u);
        n = max(0, min(n, a.lim));
    }
    const int P = a.page;
    auto page_of = [&](int p) { return a.lg_page >= 0 ? p >> a.lg_page : p / P; };
    const int pages = n > 0 ? page_of(n - 1) + 1 : 0;
    const int first = page_of(max(n - a.recent, 0));       // (recent 0: a last page that is not full stays)
    const int head = min(page_of(a.sinks) + (a.sinks - page_of(a.sinks) * P > 0), first);
    const int fixed = head * P + (n - first * P);
    const int more = min(max(page_of(max(budget - fixed, 0)), 0), first - head);
    const bool some = n > budget && more < first - head;   // some pages leave

    const float* const scores = a.scores + (int64_t)r * a.scores_ld;
    const int32_t* const table = a.table + (int64_t)r * a.ld;
    const int32_t* const positions = a.positions ? a.positions + (int64_t)r * a.ld : nullptr;
    float* const scores_out = a.scores_out + (int64_t)r * a.scores_ld;
    int32_t* const table_out = a.table_out + (int64_t)r * a.ld;
    int32_t* const positions_out = a.positions ? a.positions_out + (int64_t)r * a.ld : nullptr;

    // The first round of moves: its loads need not wait for the selection.
    float x[kEach];
    int slot[kEach], at[kEach];
    auto fetch = [&](int64_t p0) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t p = p0 + e * kThreads;
            if (p >= n) continue;
            x[e] = scores[p];
            slot[e] = table[p];
            if (positions) at[e] = positions[p];
        }
    };
    const int64_t mine0 = (int64_t)c * kThreads * kEach + tid;
    fetch(mine0);
    const int S = (pages + C - 1) / C;                     // pages of a share
    const int p0 = min(c * S, pages), np = min(S, pages - p0);       // this CTA's
    if (some) {
        if (P > 1) {
            for (int i = tid; i < np; i += kThreads) share[i] = 0;
            __syncthreads();
        }
        const int t1 = min(n, (p0 + np) * P);
#pragma unroll 4
        for (int t = p0 * P + tid; t < t1; t += kThreads) {
            const uint32_t k = order_of(scores[t]);
            if (P == 1)
                share[t - p0] = k;
            else
                atomicMax(&share[page_of(t) - p0], k);
        }
        for (int i = tid; i < kCopies * kCopyStride; i += kThreads) hist[i] = 0;
        __syncthreads();
        // lowest score that stays, and how many of those at it
        uint32_t low = 0xffffffffu, mask = 0, found = 0;
        int need = 0;
        if (more > 0) {
            int k = more;
            const int m0 = max(head - p0, 0), m1 = min(first - p0, np);
            for (int pass = 0; pass < 4; ++pass) {
                const int shift = 24 - 8 * pass;
                for (int i = m0 + tid; i < m1; i += kThreads) {
                    const uint32_t y = share[i];
                    if ((y & mask) == found) atomicAdd(&hist[(lane & (kCopies - 1)) * kCopyStride + ((y >> shift) & 255u)], 1u);
                }
                __syncthreads();
                uint32_t v = 0, upto = 0;            // pages at digit 255 - tid; and at those above, of this warp
                if (tid < 256) {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        v += hist[i * kCopyStride + 255 - tid];
                        hist[i * kCopyStride + 255 - tid] = 0;
                    }
                }
                if (tid < 256) counts[pass & 1][tid] = v;
                cl.sync();
                if (tid < 256) {
                    v = 0;
#pragma unroll
                    for (int b = 0; b < C; ++b) v += cl.map_shared_rank(counts[pass & 1], b)[tid];
                    upto = v;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += y;
                    }
                    if (lane == 31) warp_sums[warp] = upto;
                }
                __syncthreads();
                if (tid < 256) {
                    uint32_t above = upto - v;
                    for (int w = 0; w < warp; ++w) above += warp_sums[w];
                    if (above < (uint32_t)k && above + v >= (uint32_t)k) choice = make_uint3(255 - tid, above, v);
                }
                __syncthreads();
                const uint32_t digit = choice.x, above = choice.y, size = choice.z;
                k -= (int)above;
                found |= digit << shift;
                mask |= 255u << shift;
                low = found;
                need = k;
                if (size == (uint32_t)k && found > 0) {    // all of these stay: no further digit matters
                    low = found - 1;
                    need = 0;
                    break;
                }
            }
        }
        // number the kept pages: warps take runs of their CTA's share
        const int run = ((np + kWarps - 1) / kWarps + 31) & ~31;
        const int r0 = min(warp * run, np), r1 = min(r0 + run, np);
        auto sure = [&](int i) { return i < r1 && (p0 + i < head || p0 + i >= first || share[i] > low); };
        auto equal = [&](int i) { return i < r1 && p0 + i >= head && p0 + i < first && share[i] == low; };
        uint2 mine = make_uint2(0, 0);
        for (int i = r0; i < r1; i += 32) {
            mine.x += __popc(__ballot_sync(0xffffffffu, sure(i + lane)));
            mine.y += __popc(__ballot_sync(0xffffffffu, equal(i + lane)));
        }
        if (lane == 0) warp_counts[warp] = mine;
        __syncthreads();
        uint2 w = warp_counts[lane];
        const uint2 own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) {
                w.x += x;
                w.y += y;
            }
        }
        if (tid == 31) cta_counts = w;
        uint32_t surely = __shfl_sync(0xffffffffu, w.x - own.x, warp), equals = __shfl_sync(0xffffffffu, w.y - own.y, warp);
        cl.sync();
        uint2 o = lane < c ? *cl.map_shared_rank(&cta_counts, lane) : make_uint2(0, 0);
#pragma unroll
        for (int i = 8; i > 0; i >>= 1) {            // (the CTAs before this one: at most 15)
            o.x += __shfl_xor_sync(0xffffffffu, o.x, i);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, i);
        }
        surely += __shfl_sync(0xffffffffu, o.x, 0);
        equals += __shfl_sync(0xffffffffu, o.y, 0);
        const uint32_t below = (1u << lane) - 1u;
        for (int i = r0; i < r1; i += 32) {
            const bool s = sure(i + lane), e = equal(i + lane);
            const uint32_t bs = __ballot_sync(0xffffffffu, s), be = __ballot_sync(0xffffffffu, e);
            const uint32_t before = equals + __popc(be & below);       // pages at the lowest score before this one
            const int place = (int)(surely + __popc(bs & below) + min(before, (uint32_t)need));
            __syncwarp();
            if (i + lane < r1) share[i + lane] = s || (e && before < (uint32_t)need) ? (uint32_t)place : ~(uint32_t)place;
            surely += __popc(bs);
            equals += __popc(be);
        }
        cl.sync();
    }
    const int left = some ? n - (first - head - more) * P : n;
    if (c == 0 && tid == 0) {
        a.lens_out[r] = left;
        if (a.count) a.count[r] = n - left;
        if (a.evicted && n - left > a.evicted_ld) atomicOr(a.err, 2u);
    }
    if (!some && a.in_place && scores == scores_out && table == table_out && positions == positions_out) return;
    // page / S, exactly: pages and S below 2^20
    const uint64_t inv = S > 0 ? ((1ull << 40) + S - 1) / S : 0;
    for (int64_t q0 = mine0, base = 0; base < n; base += (int64_t)C * kThreads * kEach, q0 += (int64_t)C * kThreads * kEach) {
        if (base > 0) fetch(q0);
        int to[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t p = q0 + e * kThreads;
            to[e] = (int)p;
            if (some && p < n) {
                const int page = page_of((int)p), owner = (int)((page * inv) >> 40);
                const int place = (int)cl.map_shared_rank(share, owner)[page - owner * S];
                const int rest = (int)p - page * P;
                // (a page that leaves: its place among those, from the end of the ints on)
                to[e] = place >= 0 ? place * P + rest : ~((page - ~place) * P + rest);
            }
        }
        if (some && a.in_place) cl.sync();
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t p = q0 + e * kThreads;
            if (p >= n) continue;
            if (to[e] >= 0) {
                scores_out[to[e]] = x[e];
                table_out[to[e]] = slot[e];
                if (positions) positions_out[to[e]] = at[e];
            } else if (a.evicted && ~to[e] < a.evicted_ld) {
                a.evicted[(int64_t)r * a.evicted_ld + ~to[e]] = slot[e];
            }
            if (p >= left) {
                scores_out[p] = 0.f;
                table_out[p] = -1;
                if (positions) positions_out[p] = -1;
            }
        }
    }
    if (some) cl.sync();               // (others may still read this CTA's share)
}

int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return SGL_OK;
    sgl::set_cuda_error(static_cast<int>(e));
    return SGL_ERR_CUDA;
}

template <class Kernel>
int launch(Kernel* kernel, sgl::PerDevice& ready, const EvictArgs& a, int T, int B, int C, int64_t pages, cudaStream_t s) {
    if (const int e = ready_here(ready, [&] {
            if (const int e2 = large_smem(kernel, kMaxShare * 4 + 32)) return e2;
            return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        }))
        return cuda_status(static_cast<cudaError_t>(e));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3((unsigned)T);
    cfg.dynamicSmemBytes = (size_t)((pages + C - 1) / C + 8) / 8 * 32;     // (whole groups of eight)
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace

extern "C" {

int sgl_kv_evict(const sgl_evict_params* params, const float* scores, int64_t scores_ld, const int32_t* req_to_token,
                 int64_t ld, const int32_t* positions, const int32_t* lens, const int32_t* budgets, float* scores_out,
                 int32_t* table_out, int32_t* positions_out, int32_t* lens_out, int32_t* evicted, int64_t evicted_ld,
                 int32_t* evicted_count, void* workspace, size_t ws_bytes, sgl_stream_t stream) {
    if (!params || params->batch < 0 || params->page_size < 1 || params->sinks < 0 || params->recent < 0)
        return SGL_ERR_INVALID_ARG;
    if (ld < 0 || scores_ld < 0 || evicted_ld < 0) return SGL_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % sgl::kWsAlign) != 0 || ws_bytes < sgl::kWsAlign)
        return SGL_ERR_WORKSPACE;
    if (params->batch == 0) return SGL_OK;
    if (!lens || !budgets || !lens_out || !positions != !positions_out) return SGL_ERR_INVALID_ARG;
    const int64_t lim = std::min(ld, scores_ld);
    if (lim > 0 && (!scores || !req_to_token || !scores_out || !table_out)) return SGL_ERR_INVALID_ARG;
    const int P = params->page_size;
    const int64_t pages = (lim + P - 1) / P;
    if (lim > INT32_MAX / 2 || P > INT32_MAX / 2 || pages > (int64_t)kMaxCluster * kMaxShare) return SGL_ERR_UNSUPPORTED;
    EvictArgs a{};
    a.scores = scores;
    a.table = req_to_token;
    a.positions = positions;
    a.lens = lens;
    a.budgets = budgets;
    a.scores_out = scores_out;
    a.table_out = table_out;
    a.positions_out = positions_out;
    a.lens_out = lens_out;
    a.evicted = evicted;
    a.count = evicted_count;
    a.scores_ld = scores_ld;
    a.ld = ld;
    a.evicted_ld = evicted_ld;
    a.err = static_cast<uint32_t*>(workspace);
    a.page = P;
    a.lg_page = (P & (P - 1)) == 0 ? 31 - __builtin_clz(P) : -1;
    a.sinks = std::min<int32_t>(params->sinks, INT32_MAX / 2);
    a.recent = std::min<int32_t>(params->recent, INT32_MAX / 2);
    a.lanes = a.lg_page >= 0 ? std::min(P, 32) : 1;
    a.lim = (int)lim;
    a.in_place = scores == scores_out || req_to_token == table_out || (positions && positions == positions_out);
    // Rows of up to 2048 positions: a CTA of 256 threads; longer ones: 1024 threads
    // on 8192 positions each, up to 16 CTAs; and longer still, rounds of moves.
    static sgl::PerDevice ready256, ready1024, ready_long;
    auto s = reinterpret_cast<cudaStream_t>(stream);
    const int B = params->batch;
    int C = 1;
    if (lim <= 256 * kEach) return launch(evict_kernel<256>, ready256, a, 256, B, C, pages, s);
    auto share = [&] { return std::min((pages + C - 1) / C * P, lim); };     // positions of a CTA
    while (C < kMaxCluster && share() > 1024 * kEach) C *= 2;
    if ((int64_t)B * C > INT32_MAX) return SGL_ERR_UNSUPPORTED;
    if (share() <= 1024 * kEach) return launch(evict_kernel<1024>, ready1024, a, 1024, B, C, pages, s);
    return launch(evict_long_kernel, ready_long, a, 1024, B, C, pages, s);
}

}  // extern "C"
