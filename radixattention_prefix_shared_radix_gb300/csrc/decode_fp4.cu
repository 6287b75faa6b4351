// Decode attention over a 4-bit cache (SGL_DTYPE_BF16_FP4KV): work items, tiles
// and merge as in decode_fused.cu, streams of its own.
//
// At 4.5 bits a value a token's K and V of 8 heads of 128 are 1152 bytes
// instead of 4096, so per byte the streams do 3.5 times the conversions and
// products of the bf16 ones, and per token the copies are as many.  What
// differs from decode_fused.cu, and why:
//   * TMA gathers of four rows instead of a bulk copy per row.  Measured on
//     GB300 (random 576-byte rows, all SMs): two warps per SM issuing gathers
//     move 7.6 TB/s, four / eight warps of bulk copies 6.4 / 7.1.  The price
//     is that rows land back to back (no padding): bank conflicts are kept at
//     two ways by the order in which the MMA rows take the positions (pi16).
//   * Steps of 32 positions, and a running maximum that a step only has to
//     vote on, so that barriers and shuffles are paid half as often or not at
//     all.
//   * Two streaming CTAs per SM, 16 consumer warps in all.  A consumer warp is
//     a chain of conversion, scaling and product that issues an instruction
//     every four to five clocks; eight of them (one CTA of 12 warps with up to
//     168 registers, which also converted a head's codes once for 16 query
//     rows) left the issue slots 44% used and took 69 us for what the copies
//     alone do in 45.
//   * The tiles (shared prefixes) are a launch of their own, because their
//     roles need 128 registers a thread.  The streams are launched behind it
//     and start at once on the SMs that it leaves free.
//
// Streaming roles (10 warps): 0 lookup, 1 producer, 2-9 consumers (one KV head
// each for up to 8 query rows, two warps per head for up to 16).
//
// Consumer step (mma.sync m16n8k16, f16 in, fp32 acc), per 16 positions:
//   S^T [16 pos x 8 rows] = K [16 x d] . Q^T,  O^T [d x 8 rows] += V^T . P^T
// Codes go from shared memory into MMA fragments without another trip: the
// contraction of S is over d, so lane (g, t) takes the d/4 codes from (d/4) t
// of K rows g and g + 8 as its k-slots, two scales (one for d = 64) per row
// among them; in O^T, m-tile i rows g and g + 8 stand for elements (d/8) g +
// 2i and + 1, so the lane needs the d/8 codes from (d/8) g of four V rows --
// one block of 16 with one scale -- whose nibbles are paired across rows with
// two logic operations before the conversion.  A value costs half a
// conversion and half a packed multiplication (its scale).
// Conversions, packed multiplications and integer operations each run at 64
// lanes per clock and SM, mma.sync at one m16n8k16 per two clocks (measured).
// Measured: 64 requests of 1 to 8192 tokens (273 MB, 40 us at the copy's rate)
// 57.1 us.  Start and merge take 8 of the 17 above that.  In between an SM's
// two streams take 0.032 us a position (8 heads of 128) where the copies alone
// need 0.026, and no unit is full: issue slots 57%, integer pipe 51%, memory
// 61%, 28% of the warps that an SM can hold.  What is left is the latency of a
// consumer's chain from load to product: without the multiplications by scales
// (timing only) it is 4.7 us shorter, without the conversions 0.6.  One request
// of 180 tokens: 7.0 us, 2.6 of them the merge.

#include <cudaTypedefs.h>

#include "decode_stream.cuh"
#include "merge.cuh"

namespace sgl {
namespace {

constexpr int kHB = kDecHeadBlock;          // consumer warps
constexpr int kNP = 32;                     // KV positions per step
constexpr int kQuads = kNP / 4;             // gathers per pool and step
constexpr int kLookup = 0;
constexpr int kProducer = 1;
constexpr int kFirstConsumer = 2;
constexpr int kStreamThreads = 32 * (kFirstConsumer + kHB);
constexpr int kStreamCtas = 2;              // per SM
using Ent = SlotEntry<kNP>;

// the tile roles: 15 warps (10 of them gather), three K/V stages and the staging area
template <int D>
using Fp4Cfg = TcCfg<D, true, 1, 3, 10, 128, 2, kKvFp4>;

// bytes of a piece's row (its block of up to `heads` heads), as the gathers copy them
template <int D>
__host__ __device__ constexpr int fp4_box_bytes(int hkv, int heads) {
    return fp4_row_bytes(hkv < heads ? hkv : heads, D);
}

template <int D>
struct Fp4Layout {
    static constexpr int BOX = fp4_box_bytes<D>(kHB, kHB);       // the widest row
    static constexpr int QP = (4 * BOX + 127) / 128 * 128;       // a quad of rows (TMA destinations: 128-byte aligned)
    static constexpr int STAGE = 2 * kQuads * QP;                // K quads, then V quads
    static constexpr int NSF = D == 128 ? 3 : 6;                 // ring stages
    static constexpr int DESC = 64;
    static constexpr int OFF_SLOT = NSF * STAGE;
    static constexpr int OFF_DESC = OFF_SLOT + kSQ * Ent::kBytes;
    static constexpr int OFF_LREC = OFF_DESC + NSF * DESC;       // launch piece: record (32 B), members (32 B)
    static constexpr int OFF_BAR = OFF_LREC + 64;
    static constexpr int END = OFF_BAR + (2 * NSF + 2 * kSQ) * 8;
    static constexpr int TOTAL = END + 128;                      // + alignment slack
    static_assert(kStreamCtas * (TOTAL + 1024) <= 228 * 1024, "shared memory of an SM");
};

// stage descriptor: flags and the mask of the step's positions that hold data;
// a piece's first step: its fields and member requests
constexpr int kDescFlags = 0, kDescMask = 4, kDescPb = 8, kDescRows = 12, kDescNh = 16, kDescKvh = 20, kDescMem = 32;

// What a streaming CTA works with.
struct Fp4Args {
    FusedArgs f;
    int lg;                // log2 of the query heads per KV head
    float sc;              // softmax scale in base 2, times the K scale
    int box8, box4;        // bytes of a piece's row: blocks of up to 8 heads, of up to 4 (more than 8 query rows)
    int after_tiles;       // launched behind the tiles
    bf16* o;               // every request is one piece per head: results go here (and to lse), without a merge;
    float* lse;            //   else null
};

// ---------------------------------------------------------------------------
// Producer: per step waits for the slot entry and a free stage, then lane i
// gathers rows 4i .. 4i + 3 of K (i < 8) or 4i - 32 .. of V.  Rows without
// data (positions past the end, slots outside the pool) are masked by the
// consumers; a quad of them is not copied, in a mixed quad they repeat a row.
// tm: the K and V views with rows of 8 heads, then with rows of 4.
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void fp4_producer(const Fp4Args& p, const CUtensorMap* k8, const CUtensorMap* v8,
                                          const CUtensorMap* k4, const CUtensorMap* v4, uint32_t ring, uint32_t sring,
                                          uint32_t desc, uint32_t full, uint32_t empty, uint32_t sfull, uint32_t sfree,
                                          int lane) {
    using Lay = Fp4Layout<D>;
    constexpr int NS = Lay::NSF;
    uint32_t* const err = p.f.t.err;
    const int G = p.f.t.G;
    const int64_t num_slots = p.f.t.num_slots;
    const bool v = lane >= kQuads;                 // (lanes 8 .. 15)
    const int quad = lane & (kQuads - 1);
    const uint64_t kv_pol = l2_evict_first_policy();   // (read once; 58.0 -> 57.1 us on 64 requests of 1 to 8192 tokens)
    int last_armed = -1, last_arrived = -1;
    const CUtensorMap* tm = nullptr;
    uint32_t box = 0u;
    int cm = 0;                                    // end of the current piece
    for (int r = 0;; ++r) {
        const int ent = r & (kSQ - 1);
        const uint32_t eb = sring + ent * Ent::kBytes;
        if (!mbar_wait(sfull + 8 * ent, (uint32_t)(r / kSQ) & 1u)) {
            atomicOr(err, 4u);
            break;
        }
        // everything about the step is read before its stage is waited for,
        // so that its copies leave as soon as the stage is free
        const int kvh = ld_shared_s32(eb + Ent::kKvh);
        const int flags = ld_shared_s32(eb + Ent::kFlags);
        const int st = r % NS;
        const uint32_t db = desc + st * Lay::DESC;
        const uint32_t fb = full + 8 * st;
        const bool first = kvh >= 0 && (flags & kFirst) != 0;
        int pb = 0, nh = 0, nm = 0, mem = 0;
        if (first) {
            pb = ld_shared_s32(eb + Ent::kPb);
            nh = ld_shared_s32(eb + Ent::kNh);
            nm = ld_shared_s32(eb + Ent::kNm);
            cm = ld_shared_s32(eb + Ent::kCm);
            mem = lane < kDecPieceMembers ? ld_shared_s32(eb + Ent::kMem + 4 * lane) : 0;
            const bool wide = nm * G > 8;
            tm = wide ? (v ? v4 : k4) : (v ? v8 : k8);
            box = (uint32_t)(wide ? p.box4 : p.box8);
        }
        const int32_t mine = ld_shared_s32(eb + 4 * lane);
        const bool past = mine == kPastEnd || ld_shared_s32(eb + Ent::kP0) + lane >= cm;
        const bool ok = kvh >= 0 && !past && mine >= 0 && mine < num_slots;
        if (kvh >= 0 && !ok && !past) atomicOr(err, 1u);
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        int32_t row[4];
        const uint32_t qm = lane < 2 * kQuads ? (mask >> (4 * quad)) & 15u : 0u;
        const int some = 4 * quad + (qm ? __ffs(qm) - 1 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = __shfl_sync(0xffffffffu, mine, (qm >> i) & 1u ? 4 * quad + i : some);
        const uint32_t quads = __ballot_sync(0xffffffffu, qm != 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree + 8 * ent);     // every lane has read the entry
        if (!mbar_wait(empty + 8 * st, ((r / NS) & 1) ^ 1)) {
            atomicOr(err, 4u);
            break;
        }
        if (kvh < 0) {
            if (lane == 0) {
                st_shared_s32(db + kDescFlags, kEnd);
                mbar_arrive(fb);
            }
            last_arrived = r;
            break;
        }
        if (lane == 0) mbar_expect_tx_only(fb, (uint32_t)__popc(quads) * 4u * box);
        __syncwarp();
        if (qm)
            tma_gather4_hint(ring + st * Lay::STAGE + lane * Lay::QP, tm, (kvh >> 2) * (4 * fp4_head_bytes(D)) / 4, row[0],
                        row[1], row[2], row[3], fb, kv_pol);
        if (lane == 0) {
            st_shared_s32(db + kDescFlags, flags);
            st_shared_s32(db + kDescMask, (int32_t)mask);
            if (first) {
                st_shared_s32(db + kDescPb, pb);
                st_shared_s32(db + kDescRows, nm * G);
                st_shared_s32(db + kDescNh, nh);
                st_shared_s32(db + kDescKvh, kvh);
            }
        }
        if (first && lane < kDecPieceMembers) st_shared_s32(db + kDescMem + 4 * lane, mem);
        __syncwarp();
        if (lane == 0) mbar_arrive(fb);                  // the descriptor is written
        last_armed = last_arrived = r;
    }
    // this warp's copies have landed before it leaves (as in decode_fused.cu)
    const int s0 = last_arrived - NS + 1 > 0 ? last_arrived - NS + 1 : 0;
    for (int s = s0; s <= last_armed; ++s)
        if (!mbar_wait(full + 8 * (s % NS), (uint32_t)(s / NS) & 1u)) atomicOr(err, 4u);
}

// ---------------------------------------------------------------------------
// Consumer warp c: 8 query rows of one KV head of each piece
// ---------------------------------------------------------------------------

// Products and stage loads that the compiler may move (the barrier operations
// around them stay in order): D[16x8] += A[16x16] B[16x8], f16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A B
__device__ __forceinline__ void mma_f16_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(addr));
    return v;
}

// The position (0 .. 15) that MMA row m of a 16-position group takes.  A
// gathered row of 8 heads is 16 words off the banks of the one before it (d =
// 128; 8 for d = 64), so rows of both parities among every other m keep the V
// reads at two-way conflicts; neighbouring m differ in parity for the K reads.
__device__ __forceinline__ int pi16(int m) { return m ^ ((m >> 1) & 1); }

// (Registers: two CTAs of 10 warps leave 96 a thread, and a spill would go to
// L2, since the ring takes nearly all of L1: what a piece's end needs is two
// row numbers, what a step needs five addresses.)
template <int D>
__device__ __forceinline__ void fp4_consumer(const Fp4Args& p, int c, uint32_t ring, uint32_t desc, uint32_t full,
                                          uint32_t empty, uint32_t lrec, int lane) {
    using Lay = Fp4Layout<D>;
    constexpr int NS = Lay::NSF;
    constexpr int MT = D / 16;
    constexpr int KW = D / 32;                  // words of K codes per row and lane
    constexpr int VW = D / 64;                  // words of V codes per row and lane
    const int g = lane >> 2, t = lane & 3;
    const float sc = p.sc;

    uint32_t q[D / 8];
    float o[MT][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int pr0 = -1, pr1 = -1;                     // partial rows (rows of o) of this lane's two query rows
    bool have = false, active = false;
    uint32_t ka = 0u, ks = 0u, va = 0u, vs = 0u, dv = 0u;   // offsets within a stage (see below)
    auto finish_item = [&]() {
        float s0 = l0, s1 = l1;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, off);
            s1 += __shfl_xor_sync(0xffffffffu, s1, off);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int64_t prow = hh ? pr1 : pr0;
            if (prow >= 0) {
                const float ll = hh ? s1 : s0, mm = hh ? m1 : m0;
                const float inv = ll > 0.f ? p.f.t.v_scale / ll : ll;   // (0, or a NaN that is kept)
                if (p.o) {
                    uint4* dst = reinterpret_cast<uint4*>(p.o + prow * D + (D / 8) * g);
#pragma unroll
                    for (int i = 0; i < MT; i += 4)
                        dst[i / 4] = make_uint4(pack_bf16(o[i][hh] * inv, o[i][2 + hh] * inv),
                                                pack_bf16(o[i + 1][hh] * inv, o[i + 1][2 + hh] * inv),
                                                pack_bf16(o[i + 2][hh] * inv, o[i + 2][2 + hh] * inv),
                                                pack_bf16(o[i + 3][hh] * inv, o[i + 3][2 + hh] * inv));
                } else {
                    float* dst = p.f.t.po + prow * D + (D / 8) * g;
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4*>(dst + 2 * i) =
                            make_float4(o[i][hh] * inv, o[i][2 + hh] * inv, o[i + 1][hh] * inv, o[i + 1][2 + hh] * inv);
                }
                if (g == 0) (p.o ? p.lse : p.f.t.plse)[prow] = ll == 0.f ? -INFINITY : (log2f(ll) - (kPShift - mm)) * kLn2;
            }
        }
    };

    // a piece's fields and query rows: rows of nh heads from kvh on, partial rows
    // from pb on, member requests at mem in shared memory
    auto start_item = [&](int rows, int nh, int kvh, int pb, uint32_t mem) {
        const int wph = rows > 8 ? 2 : 1;   // consumer warps per head
        const int hw = c / wph, r0 = (c - hw * wph) * 8;
        active = hw < nh && r0 < rows;
        if (active) {
            // row r of a head: member r / G, query head r % G
            const int r = r0 + 2 * t, G1 = (1 << p.lg) - 1;
            auto prow = [&](int x) {
                if (x >= rows) return -1;
                return (p.o ? ld_shared_s32(mem + 4 * (x >> p.lg)) * p.f.t.Hq + ((kvh + hw) << p.lg)
                            : pb + (((x >> p.lg) * nh + hw) << p.lg)) + (x & G1);
            };
            pr0 = prow(r);
            pr1 = prow(r + 1);
            // this lane's first rows of a 16-position group: K row g (the
            // other, g + 8, lies two quads on), V row 2t (2t + 1 lies dv
            // on, 2t + 8 and 2t + 9 two quads on); the head's codes and
            // scales in them
            const uint32_t box = (uint32_t)(rows > 8 ? p.box4 : p.box8);
            const uint32_t coff = (uint32_t)fp4_code_off(hw, D), soff = (uint32_t)fp4_scale_off(hw, p.f.t.Hkv - kvh, D);
            auto roff = [&](int mrow) {
                const int x = pi16(mrow);
                return (uint32_t)((x >> 2) * Lay::QP) + (uint32_t)(x & 3) * box;
            };
            ka = roff(g) + coff + (D / 8) * t;
            ks = roff(g) + soff + (D / 64) * t;
            va = kQuads * Lay::QP + roff(2 * t) + coff + (D / 16) * g;
            vs = kQuads * Lay::QP + roff(2 * t) + soff + g * (D / 8) / 16;
            dv = roff(2 * t + 1) - roff(2 * t);
            // Q^T: row r0 + g, the lane's run of d / 4 elements in order, as f16
            const int rq = r0 + g;
            const bool ok = rq < rows;
            const int mq = ok ? ld_shared_s32(mem + 4 * (rq >> p.lg)) : 0;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.f.t.q + ((int64_t)mq * p.f.t.Hq + ((kvh + hw) << p.lg) + (rq & G1)) * D + (D / 4) * t);
            uint32_t bad = 0u;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 v = ok ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                q[4 * j] = bf16x2_to_f16x2_chk(v.x, bad);
                q[4 * j + 1] = bf16x2_to_f16x2_chk(v.y, bad);
                q[4 * j + 2] = bf16x2_to_f16x2_chk(v.z, bad);
                q[4 * j + 3] = bf16x2_to_f16x2_chk(v.w, bad);
            }
            if (bad) atomicOr(p.f.t.err, kErrQRange);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    };
    // the launch piece's are fetched while its first data is on the way
    const bool launch = (int)blockIdx.x < p.f.n_init;
    if (launch)
        start_item(ld_shared_s32(lrec + 20) << p.lg, ld_shared_s32(lrec + 28), ld_shared_s32(lrec + 12),
                   ld_shared_s32(lrec + 24), lrec + 32);

    int st = 0;
    uint32_t ph = 0u;
    for (;;) {
        if (!mbar_wait(full + 8 * st, ph)) {
            atomicOr(p.f.t.err, 4u);
            break;
        }
        const uint32_t db = desc + st * Lay::DESC;
        const int flags = ld_shared_s32(db + kDescFlags);
        const uint32_t live = (uint32_t)ld_shared_s32(db + kDescMask);    // positions of the step with data
        if (flags & kEnd) break;
        if (flags & kFirst) {
            if (have && active) finish_item();
            if (have || !launch)
                start_item(ld_shared_s32(db + kDescRows), ld_shared_s32(db + kDescNh), ld_shared_s32(db + kDescKvh),
                           ld_shared_s32(db + kDescPb), db + kDescMem);
            have = true;
        }
        const uint32_t sb = ring + st * Lay::STAGE;
        const uint32_t eb = empty + 8 * st;
        if (++st == NS) {
            st = 0;
            ph ^= 1u;
        }
        if (!active || live == 0u) {            // (an empty piece has nothing to attend to)
            __syncwarp();
            if (lane == 0) mbar_arrive(eb);
            continue;
        }
        // ---- S^T of the two position groups; in each, even and odd k-steps
        // are chains of their own (a product waits for the one before it in
        // its chain)
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t kw[2][KW], sf[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t ro = sb + (4 * u + 2 * e) * Lay::QP;
                if constexpr (D == 128) {
                    lds128(ro + ka, kw[e]);
                    sf[e] = e4m3x2_to_f16(lds_u16(ro + ks));
                } else {
                    lds64(ro + ka, kw[e]);
                    sf[e] = e4m3x2_to_f16(lds_u8(ro + ks));
                }
            }
            float s2[4];
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                // the scale of these 8 codes
                const uint32_t s0 = __byte_perm(sf[0], 0u, w < 2 ? 0x1010 : 0x3232);
                const uint32_t s1 = __byte_perm(sf[1], 0u, w < 2 ? 0x1010 : 0x3232);
                uint32_t h0[4], h1[4];
                e2m1x8_to_f16(kw[0][w], h0);
                e2m1x8_to_f16(kw[1][w], h1);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a[4] = {hmul2_u(h0[2 * k], s0), hmul2_u(h1[2 * k], s1), hmul2_u(h0[2 * k + 1], s0),
                                           hmul2_u(h1[2 * k + 1], s1)};
                    if (w == 0)
                        mma_f16_first(k ? s2 : s[u], a, q[4 * w + 2 * k], q[4 * w + 2 * k + 1]);
                    else
                        mma_f16(k ? s2 : s[u], a, q[4 * w + 2 * k], q[4 * w + 2 * k + 1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][e] += s2[e];
        }
        // ---- softmax (base 2).  The maximum that P is taken against moves
        // only when a score exceeds it by more than 8 (a factor 2^8: P stays
        // within f16), so a step needs no maximum over the lanes, only a vote
        // that nothing exceeds it.  P is taken 2^kPShift times as large (up
        // to 2^15), so that weights down to 2^-21 of the largest keep all of
        // f16's bits and smaller ones are off by 2^-32 of it at most: a long
        // context's many small weights count in full beside a large one.
        if (live != 0xffffffffu) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool ok0 = (live >> (16 * u + pi16(g))) & 1u, ok1 = (live >> (16 * u + pi16(g + 8))) & 1u;
                s[u][0] = ok0 ? s[u][0] : -INFINITY;
                s[u][1] = ok0 ? s[u][1] : -INFINITY;
                s[u][2] = ok1 ? s[u][2] : -INFINITY;
                s[u][3] = ok1 ? s[u][3] : -INFINITY;
            }
        }
        float x0 = fmaxf(fmax3f(s[0][0], s[0][2], s[1][0]), s[1][2]) * sc;
        float x1 = fmaxf(fmax3f(s[0][1], s[0][3], s[1][1]), s[1][3]) * sc;
        if (__any_sync(0xffffffffu, x0 > m0 + 8.f || x1 > m1 + 8.f)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            const float n0 = fmaxf(x0, m0), n1 = fmaxf(x1, m1);
            const float a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0);
            const float a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a1;
                o[i][2] *= a0;
                o[i][3] *= a1;
            }
        }
        const float u0 = m0 == -INFINITY ? 0.f : kPShift - m0, u1 = m1 == -INFINITY ? 0.f : kPShift - m1;
        uint32_t pf[2][2];                      // P^T fragments of the two groups
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float p00 = ex2_ftz(fmaf(s[u][0], sc, u0)), p01 = ex2_ftz(fmaf(s[u][1], sc, u1));
            const float p10 = ex2_ftz(fmaf(s[u][2], sc, u0)), p11 = ex2_ftz(fmaf(s[u][3], sc, u1));
            l0 += p00 + p10;
            l1 += p01 + p11;
            pf[u][0] = movtrans(pack_f16(p00, p01));
            pf[u][1] = movtrans(pack_f16(p10, p11));
        }
        // ---- O^T
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t vw[4][VW], sf[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t ro = sb + (4 * u + 2 * (e >> 1)) * Lay::QP + (e & 1 ? dv : 0u);
                if constexpr (D == 128)
                    lds64(ro + va, vw[e]);
                else
                    vw[e][0] = lds_u32(ro + va);
                sf[e] = lds_u8(ro + vs);
            }
            if (u == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(eb);   // the stage may be refilled
            }
            if (live != 0xffffffffu) {
                // a row without data counts nothing, whatever its scale says
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((live >> (16 * u + pi16(2 * t + (e & 1) + 8 * (e >> 1)))) & 1u)) sf[e] = 0u;
            }
            const uint32_t s01 = e4m3x2_to_f16(__byte_perm(sf[0], sf[1], 0x5540));
            const uint32_t s23 = e4m3x2_to_f16(__byte_perm(sf[2], sf[3], 0x5540));
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // byte j: elements 2j (lo) or 2j + 1 (hi) of a pair of rows
                constexpr uint32_t M = 0x0f0f0f0fu;
                uint32_t a0[4], a1[4], a2[4], a3[4];
                e2m1x8_to_f16((vw[0][w] & M) | ((vw[1][w] << 4) & ~M), a0);
                e2m1x8_to_f16(((vw[0][w] >> 4) & M) | (vw[1][w] & ~M), a1);
                e2m1x8_to_f16((vw[2][w] & M) | ((vw[3][w] << 4) & ~M), a2);
                e2m1x8_to_f16(((vw[2][w] >> 4) & M) | (vw[3][w] & ~M), a3);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a[4] = {hmul2_u(a0[j], s01), hmul2_u(a1[j], s01), hmul2_u(a2[j], s23),
                                           hmul2_u(a3[j], s23)};
                    mma_f16(o[4 * w + j], a, pf[u][0], pf[u][1]);
                }
            }
        }
    }
    if (have && active) finish_item();
}

// ---------------------------------------------------------------------------
// Tiles: CTA b runs wide items wptr[b] .. wptr[b + 1] - 1 one after another
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(Fp4Cfg<D>::kThreads, 1) decode_fp4_tiles(const __grid_constant__ FusedArgs f) {
    using TC = Fp4Cfg<D>;
    using TL = typename TC::Lay;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int w0 = __ldg(f.wptr + blockIdx.x), w1 = __ldg(f.wptr + blockIdx.x + 1);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + TL::OFF_TMEM);
    int* info = reinterpret_cast<int*>(sm + TL::OFF_INFO);
    if (tid == 0) {
        tc_init_barriers<TC>(smem_u32(sm + TL::OFF_BAR));
        mbar_fence_init();
    }
    if (warp == TC::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // what came before is complete and visible from here on, also to the
    // streams, which start only when every CTA has come to the launch below
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t tbase = *tslot;
    TcState st{0u, 0u, false};
    for (int w = w0; w < w1; ++w) {
        if (tid == 0) dec_tile_info(f.t, w, info);
        named_bar(kTileBar, TC::kThreads);
        const TileInfo ti{info[0], info[1], info[2], info[3], {info[4], 0}, {info[5], 0}, {info[6], 0}, INT_MAX, 0};
        tc_tile_run<TC>(f.t, nullptr, nullptr, nullptr, nullptr, ti, sm, tbase, st, tid);
        named_bar(kTileBar, TC::kThreads);
    }
    if (tid < 128) bulk_wait_all();   // the partial rows left as bulk copies
    tc_fence_before();
    __syncthreads();
    if (warp == TC::kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tbase));
    }
}

template <int D>
__global__ void __launch_bounds__(kStreamThreads, kStreamCtas)
    decode_fp4_streams(const __grid_constant__ Fp4Args p, const __grid_constant__ CUtensorMap k8,
                       const __grid_constant__ CUtensorMap v8, const __grid_constant__ CUtensorMap k4,
                       const __grid_constant__ CUtensorMap v4) {
    using Lay = Fp4Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const FusedArgs& f = p.f;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int NSF = Lay::NSF;
    const uint32_t ring = smem_u32(sm);            // (addresses: one register and constants)
    const uint32_t full = ring + Lay::OFF_BAR, empty = full + 8 * NSF;
    const uint32_t sfull = empty + 8 * NSF, sfree = sfull + 8 * kSQ;
    if (tid == 0) {
        for (int s = 0; s < NSF; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, kHB);
        }
        for (int e = 0; e < kSQ; ++e) {
            mbar_init(sfull + 8 * e, 33);           // the lookup lanes' cp.async + the fields
            mbar_init(sfree + 8 * e, 1);
        }
        mbar_fence_init();
    }
    // (before the dependency wait: the first copy finds the descriptors in the cache)
    if (warp == kProducer && lane < 4 && f.t.num_slots > 0) {
        const CUtensorMap* m = lane == 0 ? &k8 : lane == 1 ? &v8 : lane == 2 ? &k4 : &v4;
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
    }
    // Until the dependency wait only shared memory and the plan tables are
    // touched (see decode_fused.cu): the launch piece's record and members
    const int gw = (int)blockIdx.x;
    const uint32_t lrec = ring + Lay::OFF_LREC;
    if (warp == kLookup && gw < f.n_init) {
        const int4* rp = reinterpret_cast<const int4*>(f.narrow + gw);
        const int4 x = __ldg(rp), y = __ldg(rp + 1);
        if (lane == 0) {
            st_shared_v4(lrec, (uint32_t)x.x, (uint32_t)x.y, (uint32_t)x.z, (uint32_t)x.w);
            st_shared_v4(lrec + 16, (uint32_t)y.x, (uint32_t)y.y, (uint32_t)y.z, (uint32_t)y.w);
        }
        if (lane < kDecPieceMembers)
            st_shared_s32(lrec + 32 + 4 * lane, lane < y.y ? __ldg(f.t.members + y.x + lane) : 0);
        __syncwarp();
    }
    __syncthreads();
    // Behind the tiles, what came before them is complete already, and the
    // wait is for the tiles themselves: at the end, so that the merge, which
    // waits for this grid, comes after both.
    if (!p.after_tiles) grid_dep_wait();
    grid_dep_launch();
    const uint32_t desc = ring + Lay::OFF_DESC, sring = ring + Lay::OFF_SLOT;
    if (warp == kLookup)
        stream_lookup<kNP>(p.f, gw, lrec, sring, sfull, sfree, lane);   // up to 8 steps ahead of the copies
    else if (warp == kProducer)
        fp4_producer<D>(p, &k8, &v8, &k4, &v4, ring, sring, desc, full, empty, sfull, sfree, lane);
    else
        fp4_consumer<D>(p, warp - kFirstConsumer, ring, desc, full, empty, lrec, lane);
    if (p.after_tiles) grid_dep_wait();
}

}  // namespace

template <int D>
int launch_decode_fp4(const sgl_plan* plan, const void* q, const void* kp, const void* vp, const int32_t* r2t, int64_t ld,
                      const int32_t* seq_lens, void* o, float* lse, unsigned char* ws, float scale_log2, cudaStream_t s) {
    using Lay = Fp4Layout<D>;
    // (+ alignment slack; too much for two tile CTAs per SM: each allocates all TMEM columns)
    constexpr int kTileSmem = Fp4Cfg<D>::Lay::END + 1024 > 120 * 1024 ? Fp4Cfg<D>::Lay::END + 1024 : 120 * 1024;
    static_assert(kTileSmem <= 232448, "shared memory per CTA");
    constexpr int kMergeSmem = 216 * 1024;
    static PerDevice smem;
    if (const int e = ready_here(smem, [] {
            if (const int e0 = large_smem(decode_fp4_streams<D>, Lay::TOTAL)) return e0;
            if (const int e1 = large_smem(decode_fp4_tiles<D>, kTileSmem)) return e1;
            if (const int e2 = large_smem(decode_merge_kernel<bf16, D, 4>, kMergeSmem)) return e2;
            return large_smem(decode_merge_kernel<bf16, D, 16>, kMergeSmem);
        }))
        return e;
    const sgl_attn_params& p = plan->params;
    const int row = fp4_row_bytes(p.num_kv_heads, D);
    Fp4Args x{};
    x.box8 = fp4_box_bytes<D>(p.num_kv_heads, 8);
    x.box4 = fp4_box_bytes<D>(p.num_kv_heads, 4);
    CUtensorMap k8{}, v8{}, k4{}, v4{};
    if (plan->n_narrow > 0 && p.num_slots > 0) {
        if (const int e = tc::encode_bytes_map(kp, p.num_slots, row, x.box8, &k8)) return e;
        if (const int e = tc::encode_bytes_map(vp, p.num_slots, row, x.box8, &v8)) return e;
        if (const int e = tc::encode_bytes_map(kp, p.num_slots, row, x.box4, &k4)) return e;
        if (const int e = tc::encode_bytes_map(vp, p.num_slots, row, x.box4, &v4)) return e;
    }
    FusedArgs& f = x.f;
    TcArgs& a = f.t;
    a.q = static_cast<const bf16*>(q);
    a.kp = static_cast<const bf16*>(kp);
    a.vp = static_cast<const bf16*>(vp);
    a.r2t = r2t;
    a.ld = ld;
    a.seq_lens = seq_lens;
    a.items = reinterpret_cast<const DecItem*>(ws + plan->off_items);
    a.members = reinterpret_cast<const int32_t*>(ws + plan->off_members);
    a.po = reinterpret_cast<float*>(ws + plan->off_po);
    a.plse = reinterpret_cast<float*>(ws + plan->off_plse);
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.Hq = p.num_qo_heads;
    a.Hkv = p.num_kv_heads;
    a.G = plan->G;
    while ((1 << x.lg) < a.G) ++x.lg;
    a.num_slots = p.num_slots;
    a.scale_log2 = scale_log2;
    a.k_scale = p.k_scale;
    x.sc = scale_log2 * p.k_scale;
    a.v_scale = p.v_scale;
    a.row_bytes = row;
    f.wptr = reinterpret_cast<const int32_t*>(ws + plan->off_wptr);
    f.narrow = a.items + plan->n_wide;
    f.n_narrow = plan->n_narrow;
    f.n_init = plan->n_init;
    f.n_tile_ctas = plan->n_tile_ctas;
    f.sched = reinterpret_cast<uint32_t*>(ws + plan->off_sched);
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (plan->n_wide > 0) {
        cfg.gridDim = dim3((unsigned)plan->n_tile_ctas);
        cfg.blockDim = dim3(Fp4Cfg<D>::kThreads);
        cfg.dynamicSmemBytes = kTileSmem;
        if (const int e = (int)cudaLaunchKernelEx(&cfg, decode_fp4_tiles<D>, f)) return e;
        x.after_tiles = 1;
    }
    // (every request has a trailing piece, so there are streams whenever there are requests)
    // (when every piece is dealt at launch, a CTA for each)
    cfg.gridDim = dim3((unsigned)(plan->n_narrow <= plan->n_init ? plan->n_narrow : kStreamCtas * plan->n_ctas));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = Lay::TOTAL;
    // one piece per request and head: nothing to merge (64 requests of 64 tokens: 10.7 -> 6.6 us)
    const bool direct = plan->n_wide == 0 && plan->n_merge_entries == p.batch * p.num_kv_heads;
    if (direct) {
        x.o = static_cast<bf16*>(o);
        x.lse = lse;
    }
    if (const int e = (int)cudaLaunchKernelEx(&cfg, decode_fp4_streams<D>, x, k8, v8, k4, v4)) return e;
    if (direct) return 0;
    MergeArgs m{a.po, a.plse, reinterpret_cast<const int32_t*>(ws + plan->off_mptr),
                reinterpret_cast<const int32_t*>(ws + plan->off_ment), o, lse, a.Hq, a.Hkv, a.G};
    const int n_pairs = p.batch * a.Hkv;
    cfg.gridDim = dim3((unsigned)merge_blocks<D>(n_pairs, a.G));
    cfg.blockDim = dim3(128);
    // The merge's CTAs come to SMs as the streams leave them.  Where there are
    // more streams than SMs, the first SMs to be left would take many of them
    // and the last none, so each takes shared memory for its share of an SM (33
    // requests of 1024 tokens: 18.9 -> 16.7 us by fours, 16.4 -> 16.0 by
    // sixteens; with one stream per SM the merge gets in beside it, and the
    // share would keep it out: 12.4 -> 15.4 us for 33 of 512).  Up to four
    // entries are merged four at a time, in CTAs that need a third of the
    // registers (33 of 512 in pieces of 128: 15.3 -> 12.4; 152 of 512: 29.2 ->
    // 27.7; with eight entries sixteens are better: 12.9 -> 12.3).
    const int per = ((int)cfg.gridDim.x + plan->n_ctas - 1) / plan->n_ctas;
    cfg.dynamicSmemBytes = plan->n_narrow + plan->n_tile_ctas > plan->n_ctas ? (size_t)(kMergeSmem / per & ~1023) : 0;
    if (plan->max_entries_per_request <= 4)
        return (int)cudaLaunchKernelEx(&cfg, decode_merge_kernel<bf16, D, 4>, m, n_pairs);
    return (int)cudaLaunchKernelEx(&cfg, decode_merge_kernel<bf16, D, 16>, m, n_pairs);
}

template int launch_decode_fp4<64>(const sgl_plan*, const void*, const void*, const void*, const int32_t*, int64_t,
                                   const int32_t*, void*, float*, unsigned char*, float, cudaStream_t);
template int launch_decode_fp4<128>(const sgl_plan*, const void*, const void*, const void*, const int32_t*, int64_t,
                                    const int32_t*, void*, float*, unsigned char*, float, cudaStream_t);

}  // namespace sgl
