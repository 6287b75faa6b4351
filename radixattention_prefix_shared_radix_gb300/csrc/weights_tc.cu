// Attention weights of cached tokens from chunks of queries, on the
// 5th-generation tensor cores.
//
// The products are formed transposed, S^T = K Q^T: a row of the accumulator is a
// cached position, a column a query row (new token x query head of the KV
// head's group).  A softmax thread then has one position, and the sum over
// query rows that the operator asks for is a sum along its own columns: no
// exchange between threads, and no maximum, since the rows' log-sum-exps are
// given.  Per element: a multiply-add, an exponential, a multiply-add (packed
// in pairs but for the exponential), so that exponentials and MMAs (one k = d
// product per element) are of like size.
//
// K is the A operand and lives in TMEM (as bf16, whatever the pool holds: every
// E4M3 value, and every 4-bit value times its scale, is a bf16 value), where it
// stays for all of the item's query blocks; Q is streamed as the B operand, so
// that an MMA reads from shared memory only its N rows.
//
// An item is 256 positions (two tiles of 128 rows) of one request and KV head
// against a run of its query blocks of 128 rows; it writes 256 partial sums.
// CTAs (one per SM) take items in turn; a second launch adds the partial sums of
// a request's heads and runs in order and puts them into the scores.
//   warps 0 .. 7    softmax: tile w / 4, thread = position = TMEM lane
//   warps 8 .. 15   K: a thread takes half of a position's row of either tile
//                   from the pool (looked up an item ahead, loaded while the item
//                   before is multiplied) into TMEM, two items' rows in turn
//   warp 16         issues the MMAs (and owns TMEM)
//   warp 17         Q blocks by TMA (four stages), and the rows' log-sum-exps,
//                   in two parts, beside them (eight stages)
// All waits are bounded: one that gives up sets bit 2 of the error word, and the
// code runs to its end without hanging.

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

constexpr int kThreads = 18 * 32;
constexpr int kLoadWarp = 8, kMmaWarp = 16, kQueryWarp = 17;
constexpr int kQStages = 4, kLStages = 8;
constexpr int kMaxRows = 1 << 24;        // query rows of a call

template <int D>
struct Lay {
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int OFF_L = kQStages * QTILE;               // (-hi, -hi, factor, factor) of column pairs
    static constexpr int OFF_BAR = OFF_L + kLStages * 1024;
    static constexpr int OFF_TMEM = OFF_BAR + 40 * 8;
    static constexpr int END = OFF_TMEM + 16;
    // barriers
    static constexpr int AFULL = 0, AEMPTY = 2, SFULL = 4, SEMPTY = 6, QFULL = 8, QEMPTY = 12, LFULL = 16, LEMPTY = 24,
                         DONE = 32;
};

struct TcWeightArgs {
    WeightArgs w;
    float* partial;                      // [items, 256]
    int items, run;                      // items of the call; query blocks of an item
};

// A request's items in the order tile, run of query blocks, KV head.
struct Request {
    Asked x;
    int r, first, tiles, runs, blocks;   // first item
    int first_tile;                      // tiles of the requests before it
};

// Walks the batch 32 requests at a time, a lane per request; find() returns the
// request of an item (by_tile: of a tile).  Items must not fall from call to call.
struct Walk {
    int b = 0;                           // first request of the 32
    int64_t rows = 0;                    // query rows before them
    int items = 0, tiles = 0;            // items and tiles before them
    // this lane's request: its lengths; items and tiles up to and with it; rows before it
    int len, ext, up_items, up_tiles;
    int64_t before;
    int n_items, n_tiles, n_rows;        // of the 32
    bool filled = false;

    __device__ __forceinline__ void fill(const WeightArgs& a, int run) {
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
        const Request q = request(a, run, len, ext, before);
        up_items = q.tiles * q.runs * a.Hkv;
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
    static __device__ __forceinline__ Request request(const WeightArgs& a, int run, int len, int ext, int64_t before) {
        Request q{};
        if (len < 0 || ext < 0 || (int64_t)len + ext > a.lim || before + ext > a.n_rows) return q;
        const int ask = a.window > 0 ? min(a.window, ext) : ext;
        q.x = Asked{len + ext, ask, len + ext - ask, len, before + ext - ask};
        q.tiles = (q.x.total + 255) / 256;
        q.blocks = (ask * a.G + 127) / 128;
        q.runs = (q.blocks + run - 1) / run;
        return q;
    }
    __device__ __forceinline__ bool find(const WeightArgs& a, int run, int at, bool by_tile, Request& q) {
        for (;;) {
            if (!filled) fill(a, run);
            const uint32_t hit = __ballot_sync(0xffffffffu, by_tile ? tiles + up_tiles > at : items + up_items > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                q = request(a, run, __shfl_sync(0xffffffffu, len, l), __shfl_sync(0xffffffffu, ext, l),
                            __shfl_sync(0xffffffffu, before, l));
                q.r = b + l;
                q.first = items + __shfl_sync(0xffffffffu, up_items, l) - q.tiles * q.runs * a.Hkv;
                q.first_tile = tiles + __shfl_sync(0xffffffffu, up_tiles, l) - q.tiles;
                return true;
            }
            items += n_items;
            tiles += n_tiles;
            rows += n_rows;
            b += 32;
            filled = false;
            if (b >= a.B) return false;
        }
    }
};

struct Item {
    int at, t0, h, b0, b1, b0_1;         // first position, KV head, query blocks [b0, b1), the second tile's first
    bool two;                            // there is a second tile
    Request q;
};

// The next item from `at` on, or false; warps of every role go through the same ones.
__device__ __forceinline__ bool item_at(const TcWeightArgs& a, Walk& w, int at, Item& it) {
    if (at >= a.items || !w.find(a.w, a.run, at, false, it.q)) return false;
    const int k = at - it.q.first, tile = k % it.q.tiles, hs = k / it.q.tiles, s = hs % it.q.runs;
    it.at = at;
    it.h = hs / it.q.runs;
    it.t0 = 256 * tile;
    it.two = it.t0 + 128 < it.q.x.total;
    // a tile's rows begin with the first that sees its first position
    const int lg = 31 - __clz(a.w.G);
    auto from = [&](int t0) { return max(t0 - it.q.x.p0, 0) << lg >> 7; };
    it.b0 = max(s * a.run, from(it.t0));
    it.b1 = min((s + 1) * a.run, it.q.blocks);
    it.b0_1 = it.two ? max(it.b0, from(it.t0 + 128)) : it.b1;
    return true;
}

// (y0, y1) = (a0, a1) * (b0, b1) + (c0, c1), packed
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

// 16 consecutive TMEM columns of this thread's lane
__device__ __forceinline__ void tst16u_nw(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// an f16 pair as bf16 pairs (exact for the pools' values; NaN kept)
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
    return pack_bf16(f.x, f.y);
}

// Half a pool row of KV head h: as loaded, and as D / 4 TMEM columns (bf16 pairs).
template <int D, int KV>
struct HalfRow {
    static constexpr int RW = D * (KV == 0 ? 16 : KV == 1 ? 8 : 4) / 2 / 32;     // words
    uint32_t raw[RW], scale;
    __device__ __forceinline__ void load(const WeightArgs& a, int slot, int h, int half) {
        if (slot < 0) {
#pragma unroll
            for (int i = 0; i < RW; ++i) raw[i] = 0;
            scale = 0;
            return;
        }
        const uint8_t* row = a.kp + (int64_t)slot * a.row_bytes;
        const uint8_t* p;
        if constexpr (KV == 2) {
            p = row + fp4_code_off(h, D) + half * (RW * 4);
            const uint8_t* sf = row + fp4_scale_off(h, a.Hkv, D) + half * (D / 32);
            if constexpr (D == 128)
                scale = __ldg(reinterpret_cast<const uint32_t*>(sf));
            else
                scale = __ldg(reinterpret_cast<const uint16_t*>(sf));
        } else {
            p = row + (h * 2 + half) * (RW * 4);
        }
#pragma unroll
        for (int i = 0; i < RW / 4; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(uint32_t taddr) const {
        uint32_t y[D / 4];
        if constexpr (KV == 0) {
#pragma unroll
            for (int i = 0; i < D / 4; ++i) y[i] = raw[i];
        } else if constexpr (KV == 1) {
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                uint32_t lo, hi;
                e4m3x4_to_f16(raw[i], lo, hi);
                y[2 * i] = bf16x2_of_f16x2(lo);
                y[2 * i + 1] = bf16x2_of_f16x2(hi);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RW; ++i) {           // a word is half a block of 16
                const uint32_t sf = e4m3x2_to_f16(scale >> (8 * (i / 2)) & 0xffu), s2 = __byte_perm(sf, sf, 0x1010);
                uint32_t f[4];
                e2m1x8_to_f16(raw[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[4 * i + j] = bf16x2_of_f16x2(hmul2_u(f[j], s2));
            }
        }
        if constexpr (D == 128)
            tst32u_nw(taddr, y);
        else
            tst16u_nw(taddr, y);
    }
};

template <int D, int KV>
__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const __grid_constant__ TcWeightArgs a,
                                                                 const __grid_constant__ CUtensorMap tmq) {
    using L = Lay<D>;
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
            mbar_init(bar(L::SFULL + i), 1);
            mbar_init(bar(L::SEMPTY + i), 4);
        }
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(bar(L::QFULL + i), 1);
            mbar_init(bar(L::QEMPTY + i), 1);
        }
        for (int i = 0; i < kLStages; ++i) {
            mbar_init(bar(L::LFULL + i), 1);
            mbar_init(bar(L::LEMPTY + i), 8);
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
        // (decided for the whole warp)
        if (!__all_sync(0xffffffffu, mbar_wait(bar(b), parity))) {
            atomicOr(a.w.err, 4u);
            gave_up = true;
        }
    };
    Walk walk;
    Item it;
    if (warp >= kLoadWarp && warp < kMmaWarp) {
        // ------------------------------------------------------------ K
        const int row = 32 * (warp & 3) + lane, half = (warp - kLoadWarp) >> 2;
        const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + half * (D / 4);
        int slot[2];
        HalfRow<D, KV> k[2];
        auto lookup = [&] {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int p = it.t0 + 128 * t + row;
                slot[t] = p < it.q.x.total ? __ldg(a.w.r2t + (int64_t)it.q.r * a.w.ld + p) : 0;
                if (p >= it.q.x.total) slot[t] = -1;
                else if (slot[t] < 0 || slot[t] >= a.w.num_slots) {
                    if (half == 0) atomicOr(a.w.err, 1u);
                    slot[t] = -1;
                }
            }
        };
        auto next = [&](int at) {                    // the next item with query blocks
            while (item_at(a, walk, at, it)) {
                if (it.b0 < it.b1) return true;
                at += (int)gridDim.x;
            }
            return false;
        };
        bool have = next((int)blockIdx.x);
        if (have) lookup();
        for (uint32_t n = 0; have; ++n) {
            const bool two = it.two;
            k[0].load(a.w, slot[0], it.h, half);
            if (two) k[1].load(a.w, slot[1], it.h, half);
            have = next(it.at + (int)gridDim.x);
            if (have) lookup();
            const uint32_t ab = n & 1u;
            wait(L::AEMPTY + ab, ((n >> 1) & 1u) ^ 1u);
            if (gave_up) break;
            tc_fence_after();
            k[0].store(tl + ab * 128);
            if (two) k[1].store(tl + ab * 128 + 64);
            tst_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::AFULL + ab));
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t I = idesc_bf16(128, 128, false);
        uint32_t n = 0, qn = 0, sn[2] = {0, 0};
        for (int at = blockIdx.x; item_at(a, walk, at, it); at += gridDim.x) {
            if (it.b0 >= it.b1) continue;
            const uint32_t ab = n & 1u;
            wait(L::AFULL + ab, (n >> 1) & 1u);
            ++n;
            for (int b = it.b0; b < it.b1; ++b, ++qn) {
                const uint32_t st = qn % kQStages;
                wait(L::QFULL + st, (qn / kQStages) & 1u);
                if (gave_up) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && b < it.b0_1) continue;
                    wait(L::SEMPTY + t, (sn[t] & 1u) ^ 1u);
                    ++sn[t];
                    if (gave_up) break;
                    tc_fence_after();
                    if (lane == 0) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc_mma_tmem_a(tbase + 256 + 128 * t, tbase + ab * 128 + t * 64 + ks * 8,
                                          sdesc(sq + st * L::QTILE + (ks >> 2) * kQRegion + (ks & 3) * 32, 16, 1024), I, ks > 0);
                        tc_commit(bar(L::SFULL + t));
                    }
                    __syncwarp();
                }
                if (gave_up) break;
                if (lane == 0) {
                    tc_commit(bar(L::QEMPTY + st));
                    if (b + 1 == it.b1) tc_commit(bar(L::AEMPTY + ab));
                }
                __syncwarp();
            }
            if (gave_up) break;
        }
        // every MMA and commit has finished before this warp goes on
        if (lane == 0) tc_commit(bar(L::DONE));
        if (!mbar_wait(bar(L::DONE), 0)) atomicOr(a.w.err, 4u);
        __syncwarp();
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ Q and log-sum-exps
        const int lg = 31 - __clz(a.w.G);
        uint32_t qn = 0;
        for (int at = blockIdx.x; item_at(a, walk, at, it); at += gridDim.x) {
            float nx[4];
            // columns 4 lane .. 4 lane + 3 of block b
            auto fetch = [&](int b) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rho = 128 * b + 4 * lane + i;
                    nx[i] = -INFINITY;
                    if (rho < it.q.x.ask << lg)
                        nx[i] = __ldg(a.w.lse + (it.q.x.row + (rho >> lg)) * a.w.Hq + (it.h << lg) + (rho & (a.w.G - 1)));
                }
            };
            if (it.b0 < it.b1) fetch(it.b0);
            for (int b = it.b0; b < it.b1; ++b, ++qn) {
                const uint32_t st = qn % kQStages, ls = qn % kLStages;
                wait(L::QEMPTY + st, ((qn / kQStages) & 1u) ^ 1u);
                if (gave_up) break;
                if (lane == 0) {
                    mbar_expect_tx(bar(L::QFULL + st), L::QTILE);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_box3(sq + st * L::QTILE + x * kQRegion, &tmq, 64 * x, it.h << lg,
                                      (int)it.q.x.row + (b << 7 >> lg), bar(L::QFULL + st));
                }
                float2 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = lse_parts(nx[i]);
                if (b + 1 < it.b1) fetch(b + 1);
                wait(L::LEMPTY + ls, ((qn / kLStages) & 1u) ^ 1u);
                if (gave_up) break;
                const uint32_t to = sl + ls * 1024 + 32 * lane;
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    st_shared_v4(to + 8 * i, __float_as_uint(-y[i].x), __float_as_uint(-y[i + 1].x), __float_as_uint(y[i].y),
                                 __float_as_uint(y[i + 1].y));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::LFULL + ls));
            }
            if (gave_up) break;
        }
        // (no copy in flight when the CTA ends, also where a wait gave up)
        for (uint32_t i = qn > kQStages ? qn - kQStages : 0; gave_up && i < qn; ++i)
            mbar_wait(bar(L::QFULL + i % kQStages), (i / kQStages) & 1u);
    } else {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, row = tid & 127, lg = 31 - __clz(a.w.G);
        const uint32_t ts = tbase + 256 + 128 * t + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint64_t scale2 = pack2(a.w.scale, a.w.scale);
        uint32_t qn = 0, sn = 0;
        for (int at = blockIdx.x; item_at(a, walk, at, it); at += gridDim.x) {
            const int pos = it.t0 + 128 * t + row;
            float sum = 0.f;
            for (int b = it.b0; b < it.b1; ++b, ++qn) {
                const uint32_t ls = qn % kLStages;
                if (t == 0 || b >= it.b0_1) {
                    // columns that this position is seen by: of rows that ask, from the first that stands at it or behind
                    const int lo = max(((pos - it.q.x.p0) << lg) - 128 * b, 0), hi = min((it.q.x.ask << lg) - 128 * b, 128);
                    const bool all = __all_sync(0xffffffffu, lo <= 0) && hi == 128;
                    wait(L::LFULL + ls, (qn / kLStages) & 1u);
                    wait(L::SFULL + t, sn & 1u);
                    ++sn;
                    if (gave_up) break;
                    tc_fence_after();
                    uint64_t acc[2] = {0, 0};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[64];
                        tld64_nw(ts + 64 * half, v);
                        tld_wait();
                        if (half == 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(L::SEMPTY + t));
                        }
                        const uint32_t lp = sl + ls * 1024 + 512 * half;
                        auto terms = [&](auto masked) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                uint32_t w[4];
                                lds128(lp + 16 * j, w);
                                float x0, x1;
                                unpack2(fma2(pack2(v[2 * j], v[2 * j + 1]), scale2,
                                             pack2(__uint_as_float(w[0]), __uint_as_float(w[1]))), x0, x1);
                                x0 = ex2_ftz(x0);
                                x1 = ex2_ftz(x1);
                                if constexpr (decltype(masked)::value) {
                                    const int c = 64 * half + 2 * j;
                                    x0 = c >= lo && c < hi ? x0 : 0.f;
                                    x1 = c + 1 >= lo && c + 1 < hi ? x1 : 0.f;
                                }
                                acc[j & 1] = fma2(pack2(x0, x1), pack2(__uint_as_float(w[2]), __uint_as_float(w[3])), acc[j & 1]);
                            }
                        };
                        if (all)
                            terms(std::false_type{});
                        else
                            terms(std::true_type{});
                    }
                    float p0, p1, p2, p3;
                    unpack2(acc[0], p0, p1);
                    unpack2(acc[1], p2, p3);
                    sum += (p0 + p1) + (p2 + p3);        // (a block's sum by itself: long chains round more)
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::LEMPTY + ls));
            }
            if (gave_up) break;
            a.partial[(int64_t)at * 256 + 128 * t + row] = sum;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tbase));
    }
}

// The partial sums of a tile's heads and runs, in order, into its scores.
__global__ void __launch_bounds__(256) weights_join(const __grid_constant__ TcWeightArgs a) {
    __shared__ Request sr;
    __shared__ int found;
    const int tid = threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    if (tid < 32) {
        Walk walk;
        Request q{};
        const bool ok = walk.find(a.w, a.run, (int)blockIdx.x, true, q);
        if (tid == 0) {
            sr = q;
            found = ok;
        }
        if (blockIdx.x == 0) {           // lengths that the tables do not hold
            int64_t before = 0;
            for (int b = 0; b < a.w.B; b += 32) {
                const int r = b + tid, e = r < a.w.B ? min(max(__ldg(a.w.ext + r), 0), kMaxRows) : 0;
                int64_t s = e;
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
                    if (tid >= o) s += y;
                }
                if (r < a.w.B) asked(a.w, r, before + s - e, true);
                before += __shfl_sync(0xffffffffu, s, 31);
            }
        }
    }
    __syncthreads();
    if (!found) return;
    const Request q = sr;
    const int tile = (int)blockIdx.x - q.first_tile, pos = 256 * tile + tid;
    if (pos >= q.x.total) return;
    const int slot = __ldg(a.w.r2t + (int64_t)q.r * a.w.ld + pos);
    const int64_t at = (int64_t)q.r * a.w.scores_ld + pos;
    const bool had = a.w.in && pos < q.x.fresh;
    const float old = had ? a.w.in[at] : 0.f;
    float s = 0.f;
    const int n = q.runs * a.w.Hkv;
    if (q.first + n * q.tiles <= a.items)
        for (int i = 0; i < n; ++i) s += a.partial[((int64_t)q.first + i * q.tiles + tile) * 256 + tid];
    if (slot < 0 || slot >= a.w.num_slots) {
        s = 0.f;
        atomicOr(a.w.err, 1u);
    }
    a.w.out[at] = had ? fmaf(a.w.decay, old, s) : s;
}

template <int D, int KV>
cudaError_t run(const TcWeightArgs& a, const CUtensorMap& tmq, int ctas, cudaStream_t s) {
    constexpr int smem = Lay<D>::END + 1024;
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
// (valid ones, at most kMaxRows query rows).
TcPlan tc_plan(const sgl_attn_params* p, int window) {
    const int G = p->num_qo_heads / p->num_kv_heads;
    auto size = [&](int r, int64_t& tiles, int64_t& blocks) {
        const int64_t e = p->host_extend_lens[r], ask = window > 0 ? std::min<int64_t>(window, e) : e;
        tiles = (p->host_prefix_lens[r] + e + 255) / 256;
        blocks = (ask * G + 127) / 128;
    };
    TcPlan x{0, 0, 1};
    int64_t units = 0, tiles, blocks;
    for (int r = 0; r < p->batch; ++r) {
        size(r, tiles, blocks);
        x.tiles += tiles;
        units += tiles * blocks * p->num_kv_heads;
    }
    // four items for each SM, of at most 16 query blocks
    x.run = (int)std::min<int64_t>(std::max<int64_t>((units + 4 * 152 - 1) / (4 * 152), 1), 16);
    for (int r = 0; r < p->batch; ++r) {
        size(r, tiles, blocks);
        x.items += tiles * ((blocks + x.run - 1) / x.run) * p->num_kv_heads;
    }
    return x;
}

int launch_weights_tc(const WeightArgs& w, int kv, int d, const TcPlan& plan, float* partial, cudaStream_t s) {
    if (plan.items > INT32_MAX / 2 || plan.tiles > INT32_MAX / 2 || w.n_rows > kMaxRows) return -1;
    TcWeightArgs a{w, partial, (int)plan.items, plan.run};
    if (plan.items > 0) {
        CUtensorMap tmq{};
        if (const int e = encode_query_map(w.q, w.n_rows, w.Hq, d, w.G, 128 / w.G, &tmq)) return e;
        const int ctas = (int)std::min<int64_t>(152, plan.items);
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
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, weights_join, a);
}

}  // namespace wts
}  // namespace sgl
