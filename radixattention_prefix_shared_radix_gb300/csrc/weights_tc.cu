// Attention weights of cached tokens from chunks of queries, on the
// 5th-generation tensor cores.
//
// The products are formed transposed, S^T = K Q^T: a row of the accumulator is a
// cached position, a column a query row (new token x query head of the KV
// head's group).  A softmax thread then has one position, and the sum over
// query rows that the operator asks for is a sum along its own columns: no
// exchange between threads, and no maximum, since the rows' log-sum-exps are
// given.  Per element: a multiply-add, a product, an exponential and an addition
// (packed in pairs but for the exponential), so that exponentials and MMAs (one
// k = d product per element) are of like size.
//
// K is the A operand and lives in TMEM (as bf16, whatever the pool holds: every
// E4M3 value, and every 4-bit value times its scale, is a bf16 value), where it
// stays for all of the item's query blocks; Q is streamed as the B operand, so
// that an MMA reads from shared memory only its N rows.
//
// An item is 256 positions (two tiles of 128 rows) of one request and KV head
// against a run of its query blocks of 128 rows; CTAs (one per SM) take items in
// turn.  Two warpgroups share a block's columns, 64 each, for both tiles: a
// column's log-sum-exp, which every position needs, comes from shared memory as a
// broadcast, and a warp's broadcast costs the same 512 bytes of bandwidth
// whatever it is worth, so it is used for two positions at once.  A whole half
// block (128 scores of a thread) goes to registers before any exponential, which
// hands the accumulators back to the MMAs; the warpgroups have 168 registers a
// thread for it, taken from the others.  The two warpgroups' sums, 256 each, go
// to memory; a second launch adds those of a request's heads and runs in order
// and puts them into the scores.
//   warps 0 .. 7    softmax: columns 64 (w / 4) on, thread = TMEM lane
//   warps 8 .. 15   K: tile w / 4 - 2, rows 32 (w % 4) on, copied to shared memory an
//                   item or two ahead, and from there, converted, to TMEM, where
//                   two items' rows take turns
//   warp 16         issues the MMAs (and owns TMEM)
//   warp 17         Q blocks by TMA, and beside them the rows' log-sum-exps, which
//                   it loads a block ahead
//   warp 18         finds the items and puts them where the others read them
// All waits are bounded: one that gives up sets bit 2 of the error word, and the
// code runs to its end without hanging.
//
// 8 x 512 new tokens behind 4096, 64 heads of 128: 236 us with the join in calls
// back to back, 1240 TFLOP/s, 0.64 of the measured peak (152 us); 247 a call among
// others.  A block of 128 rows by 256
// positions is 1024 cycles of MMAs and 1024 of exponentials (32 a cycle and SM);
// it takes about 1900 (clock stamps of a softmax warp): 1350 of exponentials and
// what goes with them, then, for all warps at once, 170 until the next scores are
// seen, 190 to read them, 150 of loop and barriers.  ncu: tensor pipe and
// exponential unit 53% each, issue slots 50%, DRAM 7%.  Steps on the way: a
// warpgroup per tile, whose broadcasts of (hi, lo) log-sum-exps filled shared
// memory's bandwidth (2048 of 2800 cycles a block), 339 us; columns shared as above
// 285; items found by a warp of their own and one wait a block 252; only items
// with work numbered, so that 152 CTAs get equal shares, 235.  Without the
// product by log2 e (the log-sum-exp rounded in base 2) it takes 227, and loses
// bits of every weight.  Blocks of N = 64, which would let the warpgroups run out
// of step, cost 0.8 of the time of N = 128.  What remains at d = 128 is that two
// sets of keys and one of scores fill TMEM; at d = 64 (221 us; 122 for its
// exponentials) the keys take half as much, and 128 columns lie idle.
// Windows (one block an item): 16 x 32 rows over 1500 to 4000 tokens in 4 bits 33.0
// us, in E4M3 32.2, in bf16 44.2, about 3800 cycles an item.  An item's chain of
// copy, conversion, product, exponentials and sums has no second block to hide
// behind, and every item fetches its block of queries anew; conversion is not what
// bounds it (bf16, which needs none, takes longest, with one staged tile for each
// load warpgroup and twice the bytes; a second load warpgroup gave 0.3 us).

#include <algorithm>

#include "tc_tile.cuh"
#include "weights.cuh"

namespace sgl {
namespace tc {
int encode_query_map(const void* base, int64_t rows, int Hq, int D, int heads, int box_rows, CUtensorMap* m);
}
namespace wts {
namespace {

using namespace tc;

constexpr int kThreads = 640;
constexpr int kLoadWarp = 8, kMmaWarp = 16, kQueryWarp = 17, kItemWarp = 18;
constexpr int kReaders = 18;             // warps that go through the items
constexpr int kLStages = 8;
constexpr int kItems = 8;                // items found ahead
constexpr int kMaxRows = 1 << 24;        // query rows of a call
constexpr int kMaxTiles = 1 << 24;       // tiles x KV heads of a call
constexpr int kMaxItems = 1 << 25;       // (what tc_plan makes of these stays below it)
constexpr int kSumBlocks = 16;           // query blocks that a thread sums before it puts them away
constexpr int kItemsPerSm = 512;
// registers of a thread: 2 x 128 x 168 + 2 x 128 x 48 + 128 x 48 = the launch's 640 x 96
constexpr int kSoftmaxRegs = 168, kLoadRegs = 48, kOtherRegs = 48;

template <int D, int KV>
struct Lay {
    // a pool row of one head as staged: its bytes (4-bit rows: codes, then scales) and the stride, an odd number of 16 bytes
    static constexpr int ROW = KV == 0 ? D * 2 : KV == 1 ? D : D / 2;
    static constexpr int STRIDE = KV == 2 ? D / 2 + 16 : ROW + 16;
    static constexpr int KTILES = KV == 0 && D == 128 ? 1 : 2;   // staged tiles of each load warpgroup
    static constexpr int QSTAGES = KV == 0 && D == 128 ? 3 : 4;
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int OFF_K = QSTAGES * QTILE;
    static constexpr int OFF_L = OFF_K + 2 * KTILES * 128 * STRIDE;  // minus the log-sum-exps of a block's columns
    static constexpr int OFF_NONE = OFF_L + kLStages * 512;      // those of rows that add nothing: whether there are any; bits
    static constexpr int OFF_ITEM = OFF_NONE + kLStages * 32;
    static constexpr int OFF_BAR = OFF_ITEM + kItems * 64;
    static constexpr int OFF_TMEM = OFF_BAR + 40 * 8;
    static constexpr int END = OFF_TMEM + 16;
    // barriers
    static constexpr int AFULL = 0, AEMPTY = 2, SFULL = 4, SEMPTY = 5, QFULL = 6, QEMPTY = 10, IFULL = 14,
                         IEMPTY = IFULL + kItems, DONE = IEMPTY + kItems;
};

struct TcWeightArgs {
    WeightArgs w;
    float* partial;                      // [items, 2, 256]
    int items, run;                      // items of the call; query blocks of an item
};

// Query blocks pass a tile over until one has a row that sees its first position.
// (Int: 32 bits hold it for contexts of kMaxLen; 64 for lengths not yet checked.)
template <class Int>
__host__ __device__ __forceinline__ Int first_block(Int p0, Int t0, int lg) {
    return (t0 > p0 ? (t0 - p0) << lg : 0) >> 7;
}

// A request's items, in the order run of query blocks, tile, KV head: a tile has
// those runs that do not pass it over as a whole.
struct Request {
    Asked x;
    int r, tiles, runs, blocks;
    int head, whole;                     // items of a KV head; tiles that have every run
    int first, first_tile;               // items and tiles of the requests before it
};
// Of `tiles` tiles of 256 positions: how many have every run (they come first),
// and the items of them all.
template <class Int>
__host__ __device__ __forceinline__ int64_t items_of_head(Int p0, Int tiles, Int runs, Int run, int lg, Int* whole) {
    int64_t n = 0;
    Int w = tiles;
    for (; w > 0; --w) {
        const Int past = first_block<Int>(p0, 256 * (w - 1), lg) / run;
        if (past == 0) break;
        n += past < runs ? runs - past : 0;
    }
    *whole = w;
    return n + (int64_t)w * runs;
}

// Walks the batch 32 requests at a time, a lane per request; find() returns the
// request of an item (by_tile: of a tile).  Items must not fall from call to call.
// (Lengths may be other ones than the host planned for: sums of the items past
// the planned ones stop at kPast, so that they cannot wrap.)
constexpr int kPast = 1 << 29;
struct Walk {
    int b = 0;                           // first request of the 32
    int64_t rows = 0;                    // query rows before them
    int items = 0, tiles = 0;            // items and tiles before them
    // this lane's request: its lengths; items and tiles up to and with it; rows before it
    int len, ext, total, up_items, up_tiles;
    int64_t before;
    int n_items, n_tiles, n_rows;        // of the 32
    bool filled = false;

    __device__ __forceinline__ void fill(const TcWeightArgs& ta) {
        const WeightArgs& a = ta.w;
        const int lane = threadIdx.x & 31, r = b + lane;
        len = r < a.B ? __ldg(a.lens + r) : 0;
        ext = r < a.B ? __ldg(a.ext + r) : 0;
        const int e = min(max(ext, 0), kMaxRows);
        int se = e;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, se, o);
            if (lane >= o) se += y;
        }
        before = rows + se - e;
        n_rows = __shfl_sync(0xffffffffu, se, 31);
        const Request q = request(ta, len, ext, before);
        total = q.x.total;
        up_items = q.head * a.Hkv;
        up_tiles = q.tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, up_items, o), z = __shfl_up_sync(0xffffffffu, up_tiles, o);
            if (lane >= o) {
                up_items += y;
                up_tiles += z;
            }
        }
        n_items = __shfl_sync(0xffffffffu, up_items, 31);
        n_tiles = __shfl_sync(0xffffffffu, up_tiles, 31);
        filled = true;
    }
    static __device__ __forceinline__ Request request(const TcWeightArgs& ta, int len, int ext, int64_t before) {
        const WeightArgs& a = ta.w;
        Request q{};
        q.x = asked(a, len, ext, before);
        q.tiles = (q.x.total + 255) / 256;
        q.blocks = (q.x.ask * a.G + 127) / 128;
        q.runs = (q.blocks + ta.run - 1) / ta.run;
        const int64_t head = items_of_head<int>(q.x.p0, q.tiles, q.runs, ta.run, 31 - __clz(a.G), &q.whole);
        if (head * a.Hkv > ta.items) return Request{};       // (other lengths than the host's)
        q.head = (int)head;
        return q;
    }
    __device__ __forceinline__ bool find(const TcWeightArgs& a, int at, bool by_tile, Request& q) {
        for (;;) {
            if (!filled) fill(a);
            const uint32_t hit = __ballot_sync(0xffffffffu, by_tile ? tiles + up_tiles > at : items + up_items > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                q = request(a, __shfl_sync(0xffffffffu, len, l), __shfl_sync(0xffffffffu, ext, l),
                            __shfl_sync(0xffffffffu, before, l));
                q.r = b + l;
                q.first = items + __shfl_sync(0xffffffffu, up_items, l) - q.head * a.w.Hkv;
                q.first_tile = tiles + __shfl_sync(0xffffffffu, up_tiles, l) - q.tiles;
                return true;
            }
            items = min(items + n_items, kPast);
            tiles += n_tiles;
            rows += n_rows;
            b += 32;
            filled = false;
            if (b >= a.w.B) return false;
        }
    }
    // whether the tables hold all lengths, and what was planned all their items and tiles
    static __device__ __forceinline__ bool fits(const TcWeightArgs& a, int64_t planned_tiles) {
        Walk w;
        int64_t items = 0, tiles = 0;
        bool bad = false;
        for (; w.b < a.w.B; w.b += 32) {
            w.fill(a);
            bad |= (w.len | w.ext) != 0 && w.total == 0;
            items += w.n_items;
            tiles += w.n_tiles;
            w.rows += w.n_rows;
        }
        return !__any_sync(0xffffffffu, bad) && items <= a.items && tiles <= planned_tiles;
    }
};
static_assert((int64_t)kPast + 32 * (int64_t)kMaxItems <= INT32_MAX, "items of 32 requests, and of those before them");

// An item as its warps see it (64 bytes of shared memory).
struct alignas(16) Item {
    int at, t0, two, h;                  // -1: there are no more; first position; there is a second tile; KV head
    int b0, b1, b0_1, p0;                // query blocks [b0, b1), the second tile's first; (as in Asked) p0, ..
    int total, rows, row, r;             // .. total, query rows of a head, first query token; request
};

// Finds items, of rising numbers, by one warp; the request is kept from one to
// the next.
struct Finder {
    Walk walk;
    Request q;
    int end = 0;                         // one past the request's last item

    // item `at`, or at -1 past the last
    __device__ __forceinline__ Item item(const TcWeightArgs& a, int at) {
        Item it{};
        it.at = -1;
        if (at >= a.items) return it;
        if (at >= end) {
            if (!walk.find(a, at, false, q)) return it;
            end = q.first + q.head * a.w.Hkv;
        }
        const int lane = threadIdx.x & 31, lg = 31 - __clz(a.w.G);
        int k = at - q.first;
        it.h = k / q.head;
        k -= it.h * q.head;
        int tile, s;
        if (k < q.whole * q.runs) {
            tile = k / q.runs;
            s = k - tile * q.runs;
        } else {
            // the other tiles, 32 at a time
            k -= q.whole * q.runs;
            for (int b = q.whole;; b += 32) {
                const int past = first_block<int>(q.x.p0, 256 * (b + lane), lg) / a.run;
                const int n = b + lane < q.tiles ? max(q.runs - past, 0) : 0;
                int upto = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, upto > k);
                if (hit || b + 32 >= q.tiles) {      // (one of them holds it)
                    const int l = hit ? __ffs(hit) - 1 : 0;
                    tile = b + l;
                    s = __shfl_sync(0xffffffffu, past + k - (upto - n), l);
                    break;
                }
                k -= __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        it.at = at;
        it.t0 = 256 * tile;
        it.two = it.t0 + 128 < q.x.total;
        it.b0 = max(s * a.run, first_block<int>(q.x.p0, it.t0, lg));
        it.b1 = min((s + 1) * a.run, q.blocks);
        it.b0_1 = it.two ? max(it.b0, first_block<int>(q.x.p0, it.t0 + 128, lg)) : it.b1;
        it.p0 = q.x.p0;
        it.total = q.x.total;
        it.rows = q.x.ask << lg;
        it.row = (int)q.x.row;
        it.r = q.r;
        return it;
    }
};

// packed pairs
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 16 consecutive TMEM columns of this thread's lane
__device__ __forceinline__ void tst16u_nw(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// an f16 pair as a bf16 pair (exact for the pools' values; NaN kept)
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
    return pack_bf16(f.x, f.y);
}

// 32 elements of a staged row (a quarter of 128, half of 64) as 16 TMEM columns (bf16 pairs)
template <int D, int KV>
__device__ __forceinline__ void convert32(uint32_t row, int c, uint32_t* y) {
    if constexpr (KV == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) lds128(row + 64 * c + 16 * i, y + 4 * i);
    } else if constexpr (KV == 1) {
        uint32_t w[8];
        lds128(row + 32 * c, w);
        lds128(row + 32 * c + 16, w + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16(w[i], lo, hi);
            y[2 * i] = bf16x2_of_f16x2(lo);
            y[2 * i + 1] = bf16x2_of_f16x2(hi);
        }
    } else {
        uint32_t w[4];
        lds128(row + 16 * c, w);
        const uint32_t sf = e4m3x2_to_f16(ld_shared_u16(row + D / 2 + 2 * c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {                // a word is half a block of 16
            const uint32_t s2 = __byte_perm(sf, sf, i < 2 ? 0x1010 : 0x3232);
            uint32_t f[4];
            e2m1x8_to_f16(w[i], f);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[4 * i + j] = bf16x2_of_f16x2(hmul2_u(f[j], s2));
        }
    }
}

template <int D, int KV>
__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const __grid_constant__ TcWeightArgs a,
                                                                 const __grid_constant__ CUtensorMap tmq) {
    using L = Lay<D, KV>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sq = smem_u32(sm), sl = sq + L::OFF_L, bar0 = sq + L::OFF_BAR;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::OFF_TMEM);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::AFULL + i), 8);
            mbar_init(bar(L::AEMPTY + i), 1);
        }
        mbar_init(bar(L::SFULL), 1);
        mbar_init(bar(L::SEMPTY), 8);
        for (int i = 0; i < L::QSTAGES; ++i) {
            mbar_init(bar(L::QFULL + i), 2);
            mbar_init(bar(L::QEMPTY + i), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(bar(L::IFULL + i), 1);
            mbar_init(bar(L::IEMPTY + i), kReaders);
        }
        mbar_init(bar(L::DONE), 1);
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;
    grid_dep_wait();
    grid_dep_launch();
    bool gave_up = false;
    auto wait = [&](int b, uint32_t parity) {
        if (gave_up) return;
        // the warp polls together and decides together: lanes that polled while
        // lane 0 still had an MMA or a copy to issue could keep it from doing so
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(bar(b), parity))) {
            atomicOr(a.w.err, 4u);
            gave_up = true;
        }
    };
    // the items in turn, from the warp that finds them; false past the last
    uint32_t items_seen = 0;
    Item it;
    auto next = [&] {
        const uint32_t i = items_seen % kItems;
        wait(L::IFULL + i, (items_seen / kItems) & 1u);
        if (gave_up) return false;
        const uint32_t from = sq + L::OFF_ITEM + i * 64;
        uint32_t* w = reinterpret_cast<uint32_t*>(&it);
        lds128(from, w);
        lds128(from + 16, w + 4);
        lds128(from + 32, w + 8);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::IEMPTY + i));
        ++items_seen;
        return it.at >= 0;
    };
    if (warp < kLoadWarp) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
        const int wg = warp >> 2, row = tid & 127, lg = 31 - __clz(a.w.G);
        const uint32_t ts = tbase + 256 + 64 * wg + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint64_t scale2 = pack2(a.w.scale, a.w.scale), log2e2 = pack2(kLog2e, kLog2e);
        uint32_t qn = 0;
        while (next()) {
            float* const out = a.partial + (int64_t)it.at * 512 + 256 * wg + row;
            for (int run0 = it.b0; run0 < it.b1; run0 += kSumBlocks) {
                float sum0 = 0.f, sum1 = 0.f;
                const int run1 = min(run0 + kSumBlocks, it.b1);
                for (int b = run0; b < run1; ++b, ++qn) {
                    const bool both = b >= it.b0_1;
                    // of this warpgroup's columns, those that a position is seen by: of rows that ask, from the first that
                    // stands at it or behind
                    const int from = 128 * b + 64 * wg;
                    const int lo = ((it.t0 + row - it.p0) << lg) - from, hi = min(it.rows - from, 64);
                    // (all of them for all positions of both tiles; what stands past the context is not read)
                    const bool all = (min(it.t0 + 255, it.total - 1) - it.p0) << lg <= from && hi == 64;
                    float v0[64], v1[64];
                    wait(L::SFULL, qn & 1u);
                    if (gave_up) break;
                    tc_fence_after();
                    tld64_nw(ts, v0);
                    if (both) tld64_nw(ts + 128, v1);
                    tld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::SEMPTY));
                    const uint32_t lp = sl + qn % kLStages * 512 + 256 * wg;
                    uint64_t acc0 = 0, acc1 = 0;
                    // weights of two columns of a position, added to acc
                    auto add = [&](float s0, float s1, uint64_t m, uint64_t& acc, int c, int first, auto masked) {
                        float x0, x1;
                        unpack2(mul2(fma2(pack2(s0, s1), scale2, m), log2e2), x0, x1);
                        x0 = ex2_ftz(x0);
                        x1 = ex2_ftz(x1);
                        if constexpr (decltype(masked)::value) {
                            x0 = c >= first && c < hi ? x0 : 0.f;
                            x1 = c + 1 >= first && c + 1 < hi ? x1 : 0.f;
                        }
                        acc = add2(pack2(x0, x1), acc);
                    };
                    auto terms = [&](auto masked, auto two) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            uint32_t w[4];
                            lds128(lp + 16 * j, w);
                            const uint64_t m0 = pack2(__uint_as_float(w[0]), __uint_as_float(w[1]));
                            const uint64_t m1 = pack2(__uint_as_float(w[2]), __uint_as_float(w[3]));
                            add(v0[4 * j], v0[4 * j + 1], m0, acc0, 4 * j, lo, masked);
                            add(v0[4 * j + 2], v0[4 * j + 3], m1, acc0, 4 * j + 2, lo, masked);
                            if constexpr (decltype(two)::value) {
                                add(v1[4 * j], v1[4 * j + 1], m0, acc1, 4 * j, lo + (128 << lg), masked);
                                add(v1[4 * j + 2], v1[4 * j + 3], m1, acc1, 4 * j + 2, lo + (128 << lg), masked);
                            }
                        }
                    };
                    if (!both)
                        terms(std::true_type{}, std::false_type{});
                    else if (all)
                        terms(std::false_type{}, std::true_type{});
                    else
                        terms(std::true_type{}, std::true_type{});
                    // (a block's sum by itself: long chains round more)
                    float x, y;
                    unpack2(acc0, x, y);
                    sum0 += x + y;
                    unpack2(acc1, x, y);
                    sum1 += x + y;
                }
                if (gave_up) break;
                // (and so are those of 16 blocks: a long run's are added up in memory,
                // by this thread alone and so always in the same order)
                if (run0 == it.b0) {
                    out[0] = sum0;
                    out[128] = sum1;
                } else {
                    atomicAdd(out, sum0);
                    atomicAdd(out + 128, sum1);
                }
            }
            if (gave_up) break;
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ K
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kLoadRegs));
        const int q = warp & 3, t = (warp - kLoadWarp) >> 2;
        const uint32_t tl = tbase + ((uint32_t)(32 * q) << 16) + 64 * t;
        const uint32_t stage = sq + L::OFF_K + (t * L::KTILES * 128 + 32 * q) * L::STRIDE;       // this warp's rows of its first staged tile
        int slot = -1;
        bool more = next();
        auto lookup = [&] {                          // lane: the slot of its row of the next tile to copy
            const int p = it.t0 + 128 * t + 32 * q + lane;
            slot = -1;
            if (p < it.total) slot = __ldg(a.w.r2t + (int64_t)it.r * a.w.ld + p);
        };
        if (more) lookup();
        uint32_t copied = 0, absent = 0;             // items copied; those without this tile, by their number's low bits
        auto copy = [&] {                            // the next item's tile, as one group (empty without one)
            if (more) {
                const uint32_t to = stage + (copied % L::KTILES) * 128 * L::STRIDE;
                const bool none = t == 1 && !it.two;
                absent = (absent & ~(1u << (copied & 31u))) | (uint32_t)none << (copied & 31u);
                if (!none) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // four lanes copy a row's neighbouring pieces
                        const int r = 8 * k + (lane >> 2), s = __shfl_sync(0xffffffffu, slot, r);
                        const bool ok = s >= 0 && s < a.w.num_slots;         // (the join reports others)
                        const uint8_t* src = a.w.kp + (int64_t)(ok ? s : 0) * a.w.row_bytes
                                             + (KV == 2 ? fp4_code_off(it.h, D) : it.h * L::ROW);
                        const uint32_t dst = to + r * L::STRIDE;
#pragma unroll
                        for (int i = 0; i < (L::ROW + 63) / 64; ++i) {
                            const int piece = 4 * i + (lane & 3);
                            if (16 * piece < L::ROW) cp_async16(dst + 16 * piece, src + 16 * piece, ok);
                        }
                        if (KV == 2 && (lane & 3) == 0)
                            cp_async_small<D / 16>(dst + D / 2, a.w.kp + (int64_t)(ok ? s : 0) * a.w.row_bytes
                                                   + fp4_scale_off(it.h, a.w.Hkv, D), ok);
                    }
                }
                ++copied;
                more = next();
                if (more) lookup();
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < L::KTILES; ++i) copy();
#pragma unroll 1
        for (uint32_t n = 0; n < copied; ++n) {
            const uint32_t ab = n & 1u;
            wait(L::AEMPTY + ab, ((n >> 1) & 1u) ^ 1u);
            if (gave_up) break;
            tc_fence_after();
            cp_async_wait<L::KTILES - 1>();
            __syncwarp();
            if (!(absent >> (n & 31u) & 1u)) {
                const uint32_t from = stage + (n % L::KTILES) * 128 * L::STRIDE + lane * L::STRIDE;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t y[16];
                    convert32<D, KV>(from, c, y);
                    tst16u_nw(tl + ab * 128 + 16 * c, y);
                }
                tst_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::AFULL + ab));
            __syncwarp();
            copy();                                  // (into the tile just read)
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
        if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMA
            constexpr uint32_t I = idesc_bf16(128, 128, false);
            const uint64_t desc0 = sdesc(sq, 16, 1024);
            uint32_t n = 0, st = 0, qpar = 0, sn = 0;
            for (; next(); ++n) {
                const uint32_t ta = tbase + (n & 1u) * 128;
                for (int b = it.b0; b < it.b1; ++b, ++sn) {
                    wait(L::QFULL + st, qpar);
                    if (ld_shared_s32(sq + L::OFF_NONE + sn % kLStages * 32) && !gave_up) {
                        // Rows at -infinity add nothing, whatever they hold: zeros take their
                        // place (0 times the scale and -infinity give no weight).  Here, where
                        // keys are waited for, and not in the terms: to pass their columns over
                        // there cost 2 to 7% of every call.
                        for (int c = lane; c < 128; c += 32) {
                            const uint32_t none = ld_shared_s32(sq + L::OFF_NONE + sn % kLStages * 32 + 16 + 4 * (c & 3));
                            if (!(none >> (c >> 2) & 1u)) continue;
                            for (int x = 0; x < D / 64; ++x)
                                for (int j = 0; j < 128; j += 16)    // (whole rows: the swizzle stays within them)
                                    st_shared_v4(sq + st * L::QTILE + x * kQRegion + c * 128 + j, 0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (b == it.b0) wait(L::AFULL + (n & 1u), (n >> 1) & 1u);
                    wait(L::SEMPTY, (sn & 1u) ^ 1u);
                    if (gave_up) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t desc = desc0 + (uint64_t)(st * (L::QTILE >> 4));
                        for (int t = 0; t < (b >= it.b0_1 ? 2 : 1); ++t) {
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)
                                tc_mma_tmem_a(tbase + 256 + 128 * t, ta + t * 64 + ks * 8,
                                              desc + (uint64_t)(((ks >> 2) * kQRegion + (ks & 3) * 32) >> 4), I, ks > 0);
                        }
                        tc_commit(bar(L::SFULL));
                        tc_commit(bar(L::QEMPTY + st));
                        if (b + 1 == it.b1) tc_commit(bar(L::AEMPTY + (n & 1u)));
                    }
                    __syncwarp();
                    if (++st == L::QSTAGES) {
                        st = 0;
                        qpar ^= 1u;
                    }
                }
                if (gave_up) break;
            }
            // every MMA and commit has finished before this warp goes on
            __syncwarp();
            if (lane == 0) tc_commit(bar(L::DONE));
            __syncwarp();
            if (!mbar_wait(bar(L::DONE), 0)) atomicOr(a.w.err, 4u);
            __syncwarp();
        } else if (warp == kQueryWarp) {
            // -------------------------------------------------------- Q and log-sum-exps
            const int lg = 31 - __clz(a.w.G);
            uint32_t qn = 0;
            float nx[4];
            int b = 0;
            bool have = next();
            if (have) b = it.b0;
            auto fetch = [&] {                       // block b's columns 4 lane .. 4 lane + 3
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rho = 128 * b + 4 * lane + i;
                    nx[i] = INFINITY;                // (no row: masked)
                    if (rho < it.rows)
                        nx[i] = __ldg(a.w.lse + ((int64_t)it.row + (rho >> lg)) * a.w.Hq + (it.h << lg) + (rho & (a.w.G - 1)));
                }
            };
            if (have) fetch();
            for (; have; ++qn) {
                const uint32_t st = qn % L::QSTAGES;
                const float y[4] = {nx[0], nx[1], nx[2], nx[3]};
                const int head = it.h << lg, token = it.row + (b << 7 >> lg);
                if (++b >= it.b1) {
                    have = next();
                    b = it.b0;
                }
                if (have) fetch();
                wait(L::QEMPTY + st, ((qn / L::QSTAGES) & 1u) ^ 1u);
                if (gave_up) break;
                if (lane == 0) {
                    mbar_expect_tx(bar(L::QFULL + st), L::QTILE);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_box3(sq + st * L::QTILE + x * kQRegion, &tmq, 64 * x, head, token, bar(L::QFULL + st));
                }
                // A stage of log-sum-exps is free without a barrier of its own: block
                // qn - QSTAGES has been multiplied, so the scores of the block before
                // it have been taken, by warps that had finished the one before that,
                // and qn - kLStages lies behind.
                static_assert(kLStages >= L::QSTAGES + 2, "log-sum-exp stages");
                st_shared_v4(sl + qn % kLStages * 512 + 16 * lane, __float_as_uint(minus_lse(y[0])),
                             __float_as_uint(minus_lse(y[1])), __float_as_uint(minus_lse(y[2])), __float_as_uint(minus_lse(y[3])));
                // (bit `lane` of word i: column 4 lane + i)
                const uint32_t np = sq + L::OFF_NONE + qn % kLStages * 32;
                const int some = __any_sync(0xffffffffu, fminf(fminf(y[0], y[1]), fminf(y[2], y[3])) == -INFINITY);
                if (some) {
                    uint32_t none[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) none[i] = __ballot_sync(0xffffffffu, y[i] == -INFINITY);
                    if (lane == 0) st_shared_v4(np + 16, none[0], none[1], none[2], none[3]);
                }
                if (lane == 0) st_shared_s32(np, some);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::QFULL + st));
            }
            // (no copy in flight when the CTA ends, also where a wait gave up)
            for (uint32_t i = qn > L::QSTAGES ? qn - L::QSTAGES : 0; gave_up && i < qn; ++i)
                mbar_wait(bar(L::QFULL + i % L::QSTAGES), (i / L::QSTAGES) & 1u);
        } else if (warp == kItemWarp) {
            // -------------------------------------------------------- items
            Finder finder;
            int at = blockIdx.x;
            for (uint32_t n = 0; at >= 0; ++n) {
                const Item x = finder.item(a, at);
                const uint32_t i = n % kItems;
                wait(L::IEMPTY + i, ((n / kItems) & 1u) ^ 1u);
                if (gave_up) break;
                if (lane == 0) {
                    const uint32_t to = sq + L::OFF_ITEM + i * 64;
                    st_shared_v4(to, x.at, x.t0, x.two, x.h);
                    st_shared_v4(to + 16, x.b0, x.b1, x.b0_1, x.p0);
                    st_shared_v4(to + 32, x.total, x.rows, x.row, x.r);
                    mbar_arrive(bar(L::IFULL + i));
                }
                __syncwarp();
                at = x.at < 0 ? -1 : x.at + (int)gridDim.x;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tbase));
    }
}

// The partial sums of a tile's heads and runs, always in the same order, into its
// scores: four threads a position, a quarter of them each.
constexpr int kJoin = 4;
__global__ void __launch_bounds__(256 * kJoin, 2) weights_join(const __grid_constant__ TcWeightArgs a) {
    __shared__ Request sr;
    __shared__ int found, first, runs;   // the tile's first item of KV head 0 and its runs
    __shared__ float part[kJoin][256];
    const int tid = threadIdx.x & 255, g = threadIdx.x >> 8;
    grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x < 32) {
        Walk walk;
        Request q{};
        const bool ok = walk.find(a, (int)blockIdx.x, true, q);
        if (tid == 0) {
            sr = q;
            found = ok;
        }
        // items of the tiles before this one, 32 tiles at a time
        const int lg = 31 - __clz(a.w.G), tile = (int)blockIdx.x - q.first_tile;
        int before = 0;
        for (int t = q.whole + tid; ok && t < tile; t += 32)
            before += max(q.runs - first_block<int>(q.x.p0, 256 * t, lg) / a.run, 0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (tid == 0) {
            first = q.first + before + min(q.whole, tile) * q.runs;
            runs = ok ? max(q.runs - first_block<int>(q.x.p0, 256 * tile, lg) / a.run, 0) : 0;
        }
        __syncwarp();
    } else if (threadIdx.x < 64 && blockIdx.x == 0) {
        if (!Walk::fits(a, gridDim.x) && threadIdx.x == 32) atomicOr(a.w.err, 2u);
    }
    __syncthreads();
    if (!found) return;
    const int n = runs * a.w.Hkv, head = sr.head;
    // (a request that what was planned has no room for: its scores stay as they were)
    if (sr.first + head * a.w.Hkv > a.items || sr.first_tile + sr.tiles > (int)gridDim.x) return;
    const int pos = 256 * ((int)blockIdx.x - sr.first_tile) + tid, total = sr.x.total, r = sr.r;
    const bool mine = g == 0 && pos < total, had = mine && a.w.in && pos < sr.x.fresh;
    const int64_t at = (int64_t)r * a.w.scores_ld + pos;
    const int slot = mine ? __ldg(a.w.r2t + (int64_t)r * a.w.ld + pos) : 0;
    const float old = had ? a.w.in[at] : 0.f;
    float s = 0.f;
    if (pos < total) {
#pragma unroll 4
        for (int i = g; i < n; i += kJoin) {
            const int h = i / runs;
            const float* p = a.partial + ((int64_t)first + h * head + (i - h * runs)) * 512 + tid;
            s += p[0] + p[256];
        }
    }
    part[g][tid] = s;
    __syncthreads();
    if (!mine) return;
    s = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    if (slot < 0 || slot >= a.w.num_slots) {
        s = 0.f;
        atomicOr(a.w.err, 1u);
    }
    a.w.out[at] = had ? fmaf(a.w.decay, old, s) : s;
}

template <int D, int KV>
cudaError_t run(const TcWeightArgs& a, const CUtensorMap& tmq, int ctas, cudaStream_t s) {
    constexpr int smem = Lay<D, KV>::END + 1024;
    static_assert(smem <= 232448, "shared memory of an SM");
    static PerDevice ready;
    if (const int e = ready_here(ready, [] { return large_smem(weights_tc_kernel<D, KV>, smem); })) return (cudaError_t)e;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_tc_kernel<D, KV>, a, tmq);
}

}  // namespace

// The call's items, tiles and query blocks of an item, from the host's lengths
// (valid ones); SGL_ERR_UNSUPPORTED beyond what the kernels count.
int tc_plan(const sgl_attn_params* p, int window, TcPlan* plan) {
    const int G = p->num_qo_heads / p->num_kv_heads;
    auto size = [&](int r, int64_t& tiles, int64_t& blocks) {
        const int64_t e = p->host_extend_lens[r], ask = window > 0 ? std::min<int64_t>(window, e) : e;
        tiles = (p->host_prefix_lens[r] + e + 255) / 256;
        blocks = (ask * G + 127) / 128;
    };
    TcPlan x{0, 0, 1, target_sms(p)};
    int64_t rows = 0, units = 0, most = 1, tiles, blocks;
    for (int r = 0; r < p->batch; ++r) {
        rows += p->host_extend_lens[r];
        if ((int64_t)p->host_prefix_lens[r] + p->host_extend_lens[r] > kMaxLen || rows > kMaxRows) return SGL_ERR_UNSUPPORTED;
        size(r, tiles, blocks);
        x.tiles += tiles;
        units += tiles * blocks * p->num_kv_heads;
        most = std::max(most, blocks);
        if (x.tiles * p->num_kv_heads > kMaxTiles) return SGL_ERR_UNSUPPORTED;
    }
    // An item for each SM, of at most 16 query blocks while an SM has up to 512
    // items, beyond that as many as keep it at 512: an item's sums take 2 KB of
    // workspace however long its run is, so that what a call needs grows with its
    // positions (2 KB for 256 of them and a KV head, at least) and not with rows x
    // positions (a prompt of 131072 tokens, 64/8 heads: 84 MB; runs of 16 took 2.1 GB).
    // The longest run that rows allow, 2^20 blocks, takes a second, and a wait gives
    // up after six.
    const int64_t sms = x.sms;
    x.run = (int)std::min(std::max<int64_t>(std::clamp<int64_t>((units + sms - 1) / sms, 1, kSumBlocks),
                                            (units + kItemsPerSm * sms - 1) / (kItemsPerSm * sms)),
                          std::max<int64_t>(most, kSumBlocks));
    const int lg = 31 - __builtin_clz((unsigned)G);
    for (int r = 0; r < p->batch; ++r) {
        size(r, tiles, blocks);
        const int64_t e = p->host_extend_lens[r], ask = window > 0 ? std::min<int64_t>(window, e) : e;
        int64_t whole;
        x.items += p->num_kv_heads * items_of_head<int64_t>(p->host_prefix_lens[r] + e - ask, tiles,
                                                            (blocks + x.run - 1) / x.run, x.run, lg, &whole);
    }
    if (x.items > kMaxItems) return SGL_ERR_UNSUPPORTED;
    *plan = x;
    return SGL_OK;
}

int launch_weights_tc(const WeightArgs& w, int kv, int d, const TcPlan& plan, float* partial, cudaStream_t s) {
    TcWeightArgs a{w, partial, (int)plan.items, plan.run};
    if (plan.items > 0) {
        CUtensorMap tmq{};
        if (const int e = encode_query_map(w.q, w.n_rows, w.Hq, d, w.G, 128 / w.G, &tmq)) return e;
        const int ctas = (int)std::min<int64_t>(plan.sms, plan.items);
        cudaError_t e;
        if (d == 64)
            e = kv == 0 ? run<64, 0>(a, tmq, ctas, s) : kv == 1 ? run<64, 1>(a, tmq, ctas, s) : run<64, 2>(a, tmq, ctas, s);
        else
            e = kv == 0 ? run<128, 0>(a, tmq, ctas, s) : kv == 1 ? run<128, 1>(a, tmq, ctas, s) : run<128, 2>(a, tmq, ctas, s);
        if (e) return (int)e;
    }
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)plan.tiles);
    cfg.blockDim = dim3(256 * kJoin);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, weights_join, a);
}

}  // namespace wts
}  // namespace sgl
