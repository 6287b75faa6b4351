// Decode attention over a 4-bit cache (SGL_DTYPE_BF16_FP4KV): the persistent
// launch of decode_fused.cu -- shared prefixes on tcgen05 tiles, everything
// else streamed, then the log-sum-exp merge -- with streams of their own.
//
// At 4.5 bits a value a token's K and V of 8 heads of 128 are 1152 bytes
// instead of 4096, so per byte the streams do 3.5 times the conversions and
// products of the bf16 ones, and per token the copies are as many.  What
// differs from decode_fused.cu, and why:
//   * TMA gathers of four rows instead of a bulk copy per row.  Measured on
//     GB300 (random 576-byte rows, all SMs): two warps issuing gathers move
//     7.6 TB/s, four / eight warps of bulk copies 6.4 / 7.1.  The price is
//     that rows land back to back (no padding): bank conflicts are kept at
//     two ways by the order in which the MMA rows take the positions (pi).
//   * Steps of 32 positions, so that the softmax's shuffles, votes and the
//     barriers are paid half as often.
//   * One consumer warp per KV head for up to 16 query rows, which takes the
//     rows in one or two 8-row MMA columns: codes are converted once for both
//     (decode_fused.cu gives a head with more than 8 rows two warps, which
//     would convert everything twice).  That takes registers: 12 warps of up
//     to 168 instead of 15 of 128.
//
// Roles after the tiles (12 warps): warp 1 lookup, warps 2 and 3 producers (K
// rows, V rows), warps 4-11 consumers, one KV head each.
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

#include <cudaTypedefs.h>

#include "decode_stream.cuh"
#include "merge.cuh"

namespace sgl {
namespace {

constexpr int kHB = kDecHeadBlock;          // consumer warps = KV heads of a piece (at most)
constexpr int kNP = 32;                     // KV positions per step
constexpr int kQuads = kNP / 4;             // gathers per pool and step
constexpr int kLookup = 1;
constexpr int kFirstProducer = 2;
constexpr int kProducers = 2;               // K, V
constexpr int kFirstConsumer = 4;
constexpr int kFp4Threads = 32 * (kFirstConsumer + kHB);
using Ent = SlotEntry<kNP>;

// the tile roles: all 12 warps (7 of them gather), two K/V stages and the staging area
template <int D>
using Fp4Cfg = TcCfg<D, true, 1, 2, 7, 128, 2, kKvFp4>;
static_assert(Fp4Cfg<128>::kThreads == kFp4Threads && Fp4Cfg<64>::kThreads == kFp4Threads,
              "the tile roles take the whole CTA");

// bytes of a piece's row (its head block), as the gathers copy them
template <int D>
__host__ __device__ constexpr int fp4_box_bytes(int hkv) {
    return fp4_row_bytes(hkv < kHB ? hkv : kHB, D);
}

template <int D>
struct Fp4Layout {
    using TL = typename Fp4Cfg<D>::Lay;
    static constexpr int BOX = fp4_box_bytes<D>(kHB);            // the widest row
    static constexpr int QP = (4 * BOX + 127) / 128 * 128;       // a quad of rows (TMA destinations: 128-byte aligned)
    static constexpr int STAGE = 2 * kQuads * QP;                // K quads, then V quads
    static constexpr int SLOTW = kSQ * Ent::kBytes;
    static constexpr int DESC = 64;
    static constexpr int FIXED = 1024 + SLOTW + 12 * DESC + 64 + (2 * 12 + 2 * kSQ) * 8 + 1024;
    static constexpr int NSF0 = (232448 - FIXED) / STAGE;
    static constexpr int NSF = NSF0 > 12 ? 12 : NSF0;
    static constexpr int OFF_RING = 1024;
    static constexpr int OFF_SLOT = OFF_RING + NSF * STAGE;
    static constexpr int OFF_DESC = OFF_SLOT + SLOTW;
    static constexpr int OFF_LREC = OFF_DESC + NSF * DESC;       // launch piece: record (32 B), members (32 B)
    static constexpr int END_S = OFF_LREC + 64;
    // the streaming barriers: clear of the tile roles' area, which the rest overlaps
    static constexpr int OFF_SBAR = ((END_S > TL::END ? END_S : TL::END) + 7) / 8 * 8;
    static constexpr int END = OFF_SBAR + (2 * NSF + 2 * kSQ) * 8;
    static constexpr int TOTAL = END + 1024;                     // + alignment slack
    static_assert(NSF >= 4 && TOTAL <= 232448, "ring depth, shared memory per CTA");
    static_assert(TL::KEEP <= OFF_RING, "the ring clears the tile roles' kept area");
    static_assert(TOTAL > 116 * 1024, "one CTA per SM: tiles allocate all 512 TMEM columns");
};

// stage descriptor: position of the step, flags, mask of its positions that
// hold data; a piece's first step: its fields and member requests
constexpr int kDescP0 = 0, kDescFlags = 4, kDescMask = 8, kDescCm = 12, kDescPb = 16, kDescRows = 20, kDescNh = 24,
              kDescKvh = 28, kDescMem = 32;

// ---------------------------------------------------------------------------
// Producer warp pw (0: K, 1: V): per step waits for the slot entry and a free
// stage, then lane q < 8 gathers rows 4q .. 4q + 3.  Rows without data
// (positions past the end, slots outside the pool) are masked by the
// consumers; a quad of them is not copied, in a mixed quad they repeat a row.
// ---------------------------------------------------------------------------
template <int D>
__device__ __noinline__ void fp4_producer(const FusedArgs& f, const CUtensorMap* tm, int pw, uint32_t box, uint32_t ring,
                                          uint32_t sring, uint32_t desc, uint32_t full, uint32_t empty, uint32_t sfull,
                                          uint32_t sfree, int lane) {
    using Lay = Fp4Layout<D>;
    constexpr int NS = Lay::NSF;
    uint32_t* const err = f.t.err;
    const int G = f.t.G;
    const int64_t num_slots = f.t.num_slots;
    const bool lead = pw == 0;
    int last_armed = -1, last_arrived = -1;
    int cur_nh = 0;
    for (int r = 0;; ++r) {
        const int ent = r & (kSQ - 1);
        const uint32_t eb = sring + ent * Ent::kBytes;
        if (!mbar_wait(sfull + 8 * ent, (uint32_t)(r / kSQ) & 1u)) {
            atomicOr(err, 4u);
            break;
        }
        const int kvh = ld_shared_s32(eb + Ent::kKvh);
        const int flags = ld_shared_s32(eb + Ent::kFlags);
        const int st = r % NS;
        if (!mbar_wait(empty + 8 * st, ((r / NS) & 1) ^ 1)) {
            atomicOr(err, 4u);
            break;
        }
        const uint32_t db = desc + st * Lay::DESC;
        const uint32_t fb = full + 8 * st;
        if (kvh < 0) {
            if (lane == 0) {
                if (lead) st_shared_s32(db + kDescFlags, kEnd);
                mbar_arrive(fb);
            }
            last_arrived = r;
            __syncwarp();
            if (lane == 0) mbar_arrive(sfree + 8 * ent);
            break;
        }
        const bool first = (flags & kFirst) != 0;
        if (first) cur_nh = ld_shared_s32(eb + Ent::kNh);
        const int32_t mine = ld_shared_s32(eb + 4 * lane);
        const bool ok = mine >= 0 && mine < num_slots;
        if (lead && !ok && mine != kPastEnd) atomicOr(err, 1u);
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        int32_t row[4];
        const uint32_t qm = lane < kQuads ? (mask >> (4 * lane)) & 15u : 0u;
        if (qm) {
            const int some = ld_shared_s32(eb + 4 * (4 * lane + __ffs(qm) - 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) row[i] = (qm >> i) & 1u ? ld_shared_s32(eb + 4 * (4 * lane + i)) : some;
        }
        const uint32_t quads = __ballot_sync(0xffffffffu, qm != 0);
        if (lead && lane == 0) {
            st_shared_s32(db + kDescP0, ld_shared_s32(eb + Ent::kP0));
            st_shared_s32(db + kDescFlags, flags);
            st_shared_s32(db + kDescMask, (int32_t)mask);
            if (first) {
                st_shared_s32(db + kDescCm, ld_shared_s32(eb + Ent::kCm));
                st_shared_s32(db + kDescPb, ld_shared_s32(eb + Ent::kPb));
                st_shared_s32(db + kDescRows, ld_shared_s32(eb + Ent::kNm) * G);
                st_shared_s32(db + kDescNh, cur_nh);
                st_shared_s32(db + kDescKvh, kvh);
            }
        }
        if (lead && first && lane < kDecPieceMembers)
            st_shared_s32(db + kDescMem + 4 * lane, ld_shared_s32(eb + Ent::kMem + 4 * lane));
        __syncwarp();
        if (lane == 0) mbar_expect_tx(fb, (uint32_t)__popc(quads) * 4u * box);
        __syncwarp();
        if (qm)
            tma_gather4(ring + st * Lay::STAGE + (pw * kQuads + lane) * Lay::QP, tm,
                        (kvh >> 2) * (4 * fp4_head_bytes(D)) / 4, row[0], row[1], row[2], row[3], fb);
        last_armed = last_arrived = r;
        __syncwarp();   // every lane has read the entry
        if (lane == 0) mbar_arrive(sfree + 8 * ent);
    }
    // this warp's copies have landed before it leaves (as in decode_fused.cu)
    const int s0 = last_arrived - NS + 1 > 0 ? last_arrived - NS + 1 : 0;
    for (int s = s0; s <= last_armed; ++s)
        if (!mbar_wait(full + 8 * (s % NS), (uint32_t)(s / NS) & 1u)) atomicOr(err, 4u);
}

// ---------------------------------------------------------------------------
// Consumer warp c: KV head kvh + c of each piece
// ---------------------------------------------------------------------------

// The position (0 .. 15) that MMA row m of a 16-position group takes.  A
// gathered row is 16 words off the banks of the one before it (d = 128; 8 for
// d = 64), so rows of both parities among every other m keep the V reads at
// two-way conflicts; neighbouring m differ in parity for the K reads.
__device__ __forceinline__ int pi16(int m) { return m ^ ((m >> 1) & 1); }

struct PieceState {
    uint32_t ring, desc, full, empty;   // shared addresses
    uint32_t box;
    int cs;                             // steps consumed so far
    bool stop;
};

// All steps of one piece, from its first (whose FULL barrier has been waited
// for) to the next piece's first or the end (left for the caller), for NT
// columns of 8 query rows.
template <int D, int NT>
__device__ __forceinline__ void fp4_piece(const FusedArgs& f, PieceState& ps, int c, int lane) {
    using Lay = Fp4Layout<D>;
    constexpr int NS = Lay::NSF;
    constexpr int MT = D / 16;
    constexpr int KW = D / 32;                  // words of K codes per row and lane
    constexpr int VW = D / 64;                  // words of V codes per row and lane
    const int g = lane >> 2, t = lane & 3;
    uint32_t* const err = f.t.err;
    const int G = f.t.G, Hq = f.t.Hq, Hkv = f.t.Hkv;
    const float sc = f.t.scale_log2 * f.t.k_scale;
    const uint32_t box = ps.box;
    uint32_t db = ps.desc + (ps.cs % NS) * Lay::DESC;
    const int cm = ld_shared_s32(db + kDescCm), pb = ld_shared_s32(db + kDescPb), rows = ld_shared_s32(db + kDescRows),
              nh = ld_shared_s32(db + kDescNh), kvh = ld_shared_s32(db + kDescKvh);
    const int h = kvh + c;
    // this head's codes and scales within a piece's row
    const int coff = fp4_code_off(c, D);
    const int soff = fp4_scale_off(c, Hkv - kvh, D);
    // Q^T: row nt * 8 + g, the lane's run of d / 4 elements in order, as f16
    uint32_t q[NT][D / 8];
    uint32_t bad = 0u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rq = nt * 8 + g;
        const bool ok = rq < rows;
        const int mq = ok ? ld_shared_s32(db + kDescMem + 4 * (rq / G)) : 0;
        const uint4* src = reinterpret_cast<const uint4*>(f.t.q + ((int64_t)mq * Hq + h * G + rq % G) * D + (D / 4) * t);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const uint4 v = ok ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
            q[nt][4 * j] = bf16x2_to_f16x2_chk(v.x, bad);
            q[nt][4 * j + 1] = bf16x2_to_f16x2_chk(v.y, bad);
            q[nt][4 * j + 2] = bf16x2_to_f16x2_chk(v.z, bad);
            q[nt][4 * j + 3] = bf16x2_to_f16x2_chk(v.w, bad);
        }
    }
    if (bad) atomicOr(err, kErrQRange);
    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
    }
    // rows of this lane within a 16-position group, as stage offsets: K rows
    // g, g + 8; V rows 2t, 2t + 1, 2t + 8, 2t + 9
    auto roff = [&](int mrow) {
        const int p = pi16(mrow);
        return (uint32_t)((p >> 2) * Lay::QP) + (uint32_t)(p & 3) * box;
    };
    const uint32_t kr0 = roff(g), kr1 = roff(g + 8);
    const uint32_t vr[4] = {roff(2 * t), roff(2 * t + 1), roff(2 * t + 8), roff(2 * t + 9)};

    for (bool first = true;; first = false) {
        const int st = ps.cs % NS;
        db = ps.desc + st * Lay::DESC;
        if (!first) {
            if (!mbar_wait(ps.full + 8 * st, (ps.cs / NS) & 1)) {
                atomicOr(err, 4u);
                ps.stop = true;
                break;
            }
            if (ld_shared_s32(db + kDescFlags) & (kFirst | kEnd)) break;
        }
        const int left = cm - ld_shared_s32(db + kDescP0);      // positions of the step before the end
        uint32_t mask = (uint32_t)ld_shared_s32(db + kDescMask);
        if (left < kNP) mask &= left > 0 ? (1u << left) - 1u : 0u;
        const uint32_t sk = ps.ring + st * Lay::STAGE, sv = sk + kQuads * Lay::QP;
        ++ps.cs;
        if (mask == 0u) {   // nothing to attend to (an empty piece)
            __syncwarp();
            if (lane == 0) mbar_arrive(ps.empty + 8 * st);
            continue;
        }
        // ---- S^T
        float s[NT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t kb = sk + u * (4 * Lay::QP);
            uint32_t kw[2][KW], ksc[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t rb = kb + (e ? kr1 : kr0);
                if constexpr (D == 128) {
                    lds128(rb + coff + 16 * t, kw[e]);
                    ksc[e] = ld_shared_u16(rb + soff + 2 * t);
                } else {
                    lds64(rb + coff + 8 * t, kw[e]);
                    ksc[e] = ld_shared_u8(rb + soff + t);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][u][0] = s[nt][u][1] = s[nt][u][2] = s[nt][u][3] = 0.f;
            const uint32_t f0 = e4m3x2_to_f16(ksc[0]), f1 = e4m3x2_to_f16(ksc[1]);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                // the scale of these 8 codes
                const uint32_t s0 = __byte_perm(f0, f0, w < 2 ? 0x1010 : 0x3232);
                const uint32_t s1 = __byte_perm(f1, f1, w < 2 ? 0x1010 : 0x3232);
                uint32_t h0[4], h1[4];
                e2m1x8_to_f16(kw[0][w], h0);
                e2m1x8_to_f16(kw[1][w], h1);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t ka[4] = {hmul2_u(h0[2 * k], s0), hmul2_u(h1[2 * k], s1), hmul2_u(h0[2 * k + 1], s0),
                                            hmul2_u(h1[2 * k + 1], s1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816_f16(s[nt][u], ka, q[nt][4 * w + 2 * k], q[nt][4 * w + 2 * k + 1]);
                }
            }
        }
        // ---- softmax (base 2, lazy running maximum)
        uint32_t pf[NT][2][2];   // P^T fragments per 16 positions
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][u][e] *= sc;
                if (mask != 0xffffffffu) {
                    const bool ok0 = (mask >> (16 * u + pi16(g))) & 1u, ok1 = (mask >> (16 * u + pi16(g + 8))) & 1u;
                    s[nt][u][0] = ok0 ? s[nt][u][0] : -INFINITY;
                    s[nt][u][1] = ok0 ? s[nt][u][1] : -INFINITY;
                    s[nt][u][2] = ok1 ? s[nt][u][2] : -INFINITY;
                    s[nt][u][3] = ok1 ? s[nt][u][3] : -INFINITY;
                }
                x0 = fmax3f(x0, s[nt][u][0], s[nt][u][2]);
                x1 = fmax3f(x1, s[nt][u][1], s[nt][u][3]);
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            // the maximum that P is taken against moves only when it is
            // exceeded by more than 8 (a factor 2^8: P stays within f16)
            const bool up0 = x0 > m[nt][0] + 8.f, up1 = x1 > m[nt][1] + 8.f;
            if (__any_sync(0xffffffffu, up0 || up1)) {
                const float n0 = up0 ? x0 : m[nt][0], n1 = up1 ? x1 : m[nt][1];
                const float a0 = m[nt][0] == -INFINITY ? 0.f : exp2f(m[nt][0] - n0);
                const float a1 = m[nt][1] == -INFINITY ? 0.f : exp2f(m[nt][1] - n1);
                m[nt][0] = n0;
                m[nt][1] = n1;
                l[nt][0] *= a0;
                l[nt][1] *= a1;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[nt][i][0] *= a0;
                    o[nt][i][1] *= a1;
                    o[nt][i][2] *= a0;
                    o[nt][i][3] *= a1;
                }
            }
            const float u0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], u1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float p0 = ex2_ftz(s[nt][u][0] - u0), p1 = ex2_ftz(s[nt][u][1] - u1);
                const float p2 = ex2_ftz(s[nt][u][2] - u0), p3 = ex2_ftz(s[nt][u][3] - u1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pf[nt][u][0] = movtrans(pack_f16(p0, p1));
                pf[nt][u][1] = movtrans(pack_f16(p2, p3));
            }
        }
        // ---- O^T
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t vb = sv + u * (4 * Lay::QP);
            uint32_t vw[4][VW], vs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t rb = vb + vr[e];
                if constexpr (D == 128) {
                    lds64(rb + coff + 8 * g, vw[e]);
                    vs[e] = ld_shared_u8(rb + soff + g);
                } else {
                    vw[e][0] = (uint32_t)ld_shared_s32(rb + coff + 4 * g);
                    vs[e] = ld_shared_u8(rb + soff + (g >> 1));
                }
            }
            if (u == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(ps.empty + 8 * st);   // the stage may be refilled
            }
            if (mask != 0xffffffffu) {
                // a row without data counts nothing, whatever its scale says
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((mask >> (16 * u + pi16(2 * t + (e & 1) + 8 * (e >> 1)))) & 1u)) vs[e] = 0u;
            }
            const uint32_t s01 = e4m3x2_to_f16(vs[0] | (vs[1] << 8)), s23 = e4m3x2_to_f16(vs[2] | (vs[3] << 8));
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
                    const uint32_t va[4] = {hmul2_u(a0[j], s01), hmul2_u(a1[j], s01), hmul2_u(a2[j], s23),
                                            hmul2_u(a3[j], s23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[nt][4 * w + j], va, pf[nt][u][0], pf[nt][u][1]);
                }
            }
        }
    }
    // ---- the piece's partial rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float s0 = l[nt][0], s1 = l[nt][1];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, off);
            s1 += __shfl_xor_sync(0xffffffffu, s1, off);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = nt * 8 + 2 * t + hh;   // query row of this head: member r / G, query head r % G
            if (r < rows) {
                const int64_t prow = (int64_t)pb + ((r / G) * nh + c) * G + r % G;
                const float ll = hh ? s1 : s0, mm = m[nt][hh];
                const float inv = ll > 0.f ? f.t.v_scale / ll : 0.f;
                float* dst = f.t.po + prow * D + (D / 8) * g;
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[nt][i][hh] * inv, o[nt][i][2 + hh] * inv);
                if (g == 0) f.t.plse[prow] = ll > 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
            }
        }
    }
}

template <int D>
__device__ __noinline__ void fp4_consumer(const FusedArgs& f, int c, PieceState ps, int lane) {
    using Lay = Fp4Layout<D>;
    constexpr int NS = Lay::NSF;
    bool have = false;   // the step at ps.cs has been waited for
    while (!ps.stop) {
        const int st = ps.cs % NS;
        if (!have && !mbar_wait(ps.full + 8 * st, (ps.cs / NS) & 1)) {
            atomicOr(f.t.err, 4u);
            break;
        }
        const uint32_t db = ps.desc + st * Lay::DESC;
        const int flags = ld_shared_s32(db + kDescFlags);
        if (flags & kEnd) break;
        have = false;
        // (only a piece's first step carries the piece's head count)
        if ((flags & kFirst) && c < ld_shared_s32(db + kDescNh)) {
            if (ld_shared_s32(db + kDescRows) > 8)
                fp4_piece<D, 2>(f, ps, c, lane);
            else
                fp4_piece<D, 1>(f, ps, c, lane);
            have = true;
        } else {   // a piece without this warp's head
            ++ps.cs;
            __syncwarp();
            if (lane == 0) mbar_arrive(ps.empty + 8 * st);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kFp4Threads, 1) decode_fp4_kernel(const __grid_constant__ FusedArgs f,
                                                                    const __grid_constant__ CUtensorMap tmk,
                                                                    const __grid_constant__ CUtensorMap tmv) {
    using Lay = Fp4Layout<D>;
    using TC = Fp4Cfg<D>;
    using TL = typename TC::Lay;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Until the dependency wait only shared memory, TMEM and the plan tables
    // are touched (see decode_fused.cu).
    const int w0 = __ldg(f.wptr + blockIdx.x), w1 = __ldg(f.wptr + blockIdx.x + 1);
    const bool tiles = w1 > w0;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + TL::OFF_TMEM);
    int* info = reinterpret_cast<int*>(sm + TL::OFF_INFO);
    constexpr int NSF = Lay::NSF;
    const uint32_t sbar = smem_u32(sm + Lay::OFF_SBAR);
    const uint32_t sfull = sbar, sempty = sbar + 8 * NSF;
    const uint32_t slfull = sbar + 16 * NSF, slfree = slfull + 8 * kSQ;
    if (tid == 0) {
        if (tiles) tc_init_barriers<TC>(smem_u32(sm + TL::OFF_BAR));
        for (int s = 0; s < NSF; ++s) {
            mbar_init(sfull + 8 * s, kProducers);
            mbar_init(sempty + 8 * s, kHB);
        }
        for (int e = 0; e < kSQ; ++e) {
            mbar_init(slfull + 8 * e, 33);          // the lookup lanes' cp.async + the fields
            mbar_init(slfree + 8 * e, kProducers);
        }
        mbar_fence_init();
    }
    if (tiles && warp == TC::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tiles && tid == 0) prefetch_l1(f.t.items + w0);
    const int gw = !tiles && (int)blockIdx.x >= f.n_tile_ctas ? (int)blockIdx.x - f.n_tile_ctas : -1;
    const uint32_t lrec = smem_u32(sm + Lay::OFF_LREC);
    if (warp == kLookup && gw >= 0 && gw < f.n_init) {
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
    grid_dep_wait();
    grid_dep_launch();

    if (tiles) {
        const uint32_t tbase = *tslot;
        TcState st{0u, 0u, false};
        for (int w = w0; w < w1; ++w) {
            if (tid == 0) dec_tile_info(f.t, w, info);
            named_bar(kTileBar, TC::kThreads);
            const TileInfo ti{info[0], info[1], info[2], info[3], {info[4], 0}, {info[5], 0}, {info[6], 0}, INT_MAX, 0};
            tc_tile_run<TC>(f.t, nullptr, nullptr, nullptr, nullptr, ti, sm, tbase, st, tid);
            named_bar(kTileBar, TC::kThreads);
        }
        // the streaming areas overlap the tile roles' barriers
        if (tid == 0) tc_inval_barriers<TC>(smem_u32(sm + TL::OFF_BAR));
        named_bar(kTileBar, TC::kThreads);
    }
    const uint32_t ring = smem_u32(sm + Lay::OFF_RING);
    const uint32_t desc = smem_u32(sm + Lay::OFF_DESC);
    const uint32_t sring = smem_u32(sm + Lay::OFF_SLOT);
    const uint32_t box = (uint32_t)fp4_box_bytes<D>(f.t.Hkv);
    if (warp == kLookup) {
        stream_lookup<kNP>(f, gw, lrec, sring, slfull, slfree, lane);
    } else if (warp >= kFirstProducer && warp < kFirstConsumer) {
        const int pw = warp - kFirstProducer;
        fp4_producer<D>(f, pw ? &tmv : &tmk, pw, box, ring, sring, desc, sfull, sempty, slfull, slfree, lane);
    } else if (warp >= kFirstConsumer) {
        fp4_consumer<D>(f, warp - kFirstConsumer, PieceState{ring, desc, sfull, sempty, box, 0, false}, lane);
    }
    // the tiles' partial rows went out as bulk copies from threads 0-127
    if (tiles && tid < 128) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (tiles && warp == TC::kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(*tslot));
    }
}

}  // namespace

template <int D>
int launch_decode_fp4(const sgl_plan* plan, const void* q, const void* kp, const void* vp, const int32_t* r2t, int64_t ld,
                      const int32_t* seq_lens, void* o, float* lse, unsigned char* ws, float scale_log2, cudaStream_t s) {
    using Lay = Fp4Layout<D>;
    static const int attr = (int)cudaFuncSetAttribute(decode_fp4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      Lay::TOTAL);
    if (attr) return attr;
    const sgl_attn_params& p = plan->params;
    const int row = fp4_row_bytes(p.num_kv_heads, D);
    CUtensorMap mk{}, mv{};
    if (plan->n_narrow > 0 && p.num_slots > 0) {
        const int box = fp4_box_bytes<D>(p.num_kv_heads);
        if (const int e = tc::encode_bytes_map(kp, p.num_slots, row, box, &mk)) return e;
        if (const int e = tc::encode_bytes_map(vp, p.num_slots, row, box, &mv)) return e;
    }
    FusedArgs f{};
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
    a.num_slots = p.num_slots;
    a.scale_log2 = scale_log2;
    a.k_scale = p.k_scale;
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
    cfg.gridDim = dim3((unsigned)plan->n_ctas);
    cfg.blockDim = dim3(kFp4Threads);
    cfg.dynamicSmemBytes = Lay::TOTAL;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    int e = (int)cudaLaunchKernelEx(&cfg, decode_fp4_kernel<D>, f, mk, mv);
    if (e) return e;
    MergeArgs m{a.po, a.plse, reinterpret_cast<const int32_t*>(ws + plan->off_mptr),
                reinterpret_cast<const int32_t*>(ws + plan->off_ment), o, lse, a.Hq, a.Hkv, a.G};
    const int n_pairs = p.batch * a.Hkv;
    cfg.gridDim = dim3((unsigned)merge_blocks<D>(n_pairs, a.G));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return (int)cudaLaunchKernelEx(&cfg, decode_merge_kernel<bf16, D>, m, n_pairs);
}

template int launch_decode_fp4<64>(const sgl_plan*, const void*, const void*, const void*, const int32_t*, int64_t,
                                   const int32_t*, void*, float*, unsigned char*, float, cudaStream_t);
template int launch_decode_fp4<128>(const sgl_plan*, const void*, const void*, const void*, const int32_t*, int64_t,
                                    const int32_t*, void*, float*, unsigned char*, float, cudaStream_t);

}  // namespace sgl
