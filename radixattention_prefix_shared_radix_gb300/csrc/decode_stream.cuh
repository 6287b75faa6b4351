// What the streaming decode kernels share: their arguments, the slot ring that
// the lookup warp fills, the stage descriptors, and small helpers.
#pragma once

#include "tc_tile.cuh"

namespace sgl {
namespace {

using namespace sgldev;
using namespace tc;

struct FusedArgs {
    TcArgs t;
    const int32_t* wptr;   // [n_ctas + 1] wide items of each CTA
    const DecItem* narrow; // narrow pieces, in the order in which they are dealt and handed out
    int n_narrow;
    int n_init;            // pieces assigned at launch: streaming CTA w starts on piece w
    int n_tile_ctas;       // CTAs 0 .. n_tile_ctas-1 run the wide items first
    uint32_t* sched;       // [2] next piece to hand out, producers finished (restored at the end)
};

__device__ __forceinline__ uint32_t movtrans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// D[16x8] += A[16x16] * B[16x8], f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma16816_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t* w) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// stage descriptor flags
constexpr int kFirst = 1;   // first step of its piece: the descriptor carries the piece's fields
constexpr int kEnd = 4;     // no more pieces: the consumers stop

// slot ring: lookups ahead of the copies
constexpr int kSQ = 8;
static_assert((kSQ & (kSQ - 1)) == 0, "slot ring");
constexpr int32_t kPastEnd = INT32_MIN;   // slot of a position past the piece's end

// slot-ring entry (one looked-up step of NP positions): NP slots, then
template <int NP>
struct SlotEntry {
    static constexpr int kKvh = 4 * NP, kP0 = kKvh + 4, kFlags = kKvh + 8, kCm = kKvh + 12, kPb = kKvh + 16,
                         kNh = kKvh + 20, kNm = kKvh + 24;
    static constexpr int kMem = kKvh + 32;   // kDecPieceMembers ints: the piece's member requests (first step only)
    static constexpr int kBytes = kKvh + 64;
    static_assert(kMem + 4 * kDecPieceMembers <= kBytes, "a slot entry holds a piece's members");
};
// ---------------------------------------------------------------------------
// Lookup warp (one per CTA)
// ---------------------------------------------------------------------------
// Walks this CTA's pieces (its launch piece, whose record and members were
// loaded before the dependency wait, then pieces taken from the run-time
// counter) and fills the slot ring up to kSQ steps ahead of the producers:
// per step the NP slots (4-byte cp.async from req_to_token; positions past
// the piece's end marked), the step's first KV head, position and flags,
// and for a piece's first step its partial base, clamped end, head and
// member counts and member requests.  Each entry's barrier (SLOTFULL)
// completes when the lanes' cp.async have landed and lane 0 has written the
// fields; the producers free it (SLOTFREE).  An entry with no KV head ends
// the stream.  Global loads (the counter, records, seq_lens) stall only this
// warp, which runs ahead of the copies.
template <int NP>
__device__ __forceinline__ void stream_lookup(const FusedArgs& f, int gw, uint32_t lrec, uint32_t sring,
                                              uint32_t sfull, uint32_t sfree, int lane) {
    using Ent = SlotEntry<NP>;
    const int32_t* const r2t = f.t.r2t;
    const int32_t* const members = f.t.members;
    const int32_t* const seq_lens = f.t.seq_lens;
    const int64_t ld = f.t.ld;
    uint32_t* const err = f.t.err;
    const DecItem* const pieces = f.narrow;
    const int n_narrow = f.n_narrow;
    uint32_t* const sched = f.sched;
    const bool dealt = n_narrow <= f.n_init;   // every piece was dealt at launch: the counter is not used
    const bool launch = gw >= 0 && gw < f.n_init;
    bool timed_out = false;
    int nlook = 0;
    // one ring entry: wait for it to be free, fill it, arm its barrier.  A
    // piece's first entry also records its end clamped to seq_len (len, whose
    // load is only waited for once the slot lookups are issued)
    auto entry = [&](int kvh, int row, int p0, int e, int flags, int len, int pb, int nh, int nm, int mem) {
        const int ent = nlook & (kSQ - 1);
        const uint32_t eb = sring + ent * Ent::kBytes;
        if (!timed_out && !mbar_wait(sfree + 8 * ent, ((nlook / kSQ) & 1) ^ 1)) {
            atomicOr(err, 4u);
            timed_out = true;
        }
        if (timed_out) return;
        if (lane < NP) {
            const int p = p0 + lane;
            if (kvh >= 0 && p < e)
                cp_async4(eb + lane * 4, r2t + (int64_t)row * ld + p);
            else
                st_shared_s32(eb + lane * 4, kPastEnd);
        }
        if (lane == 0) {
            st_shared_s32(eb + Ent::kKvh, kvh);
            st_shared_s32(eb + Ent::kP0, p0);
            st_shared_s32(eb + Ent::kFlags, flags);
            if (flags & kFirst) {
                int cm = e;
                if (e > len) {   // planned beyond seq_len: mask the excess, flag it
                    atomicOr(err, 2u);
                    cm = len > p0 ? len : p0;
                }
                st_shared_s32(eb + Ent::kCm, cm);
                st_shared_s32(eb + Ent::kPb, pb);
                st_shared_s32(eb + Ent::kNh, nh);
                st_shared_s32(eb + Ent::kNm, nm);
            }
        }
        if ((flags & kFirst) && lane < kDecPieceMembers) st_shared_s32(eb + Ent::kMem + 4 * lane, mem);
        cp_async_arrive_noinc(sfull + 8 * ent);   // each lane, once its lookups have landed
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull + 8 * ent);   // the fields
        ++nlook;
    };
    bool first_piece = true;
    for (;;) {
        int row, b, e, kvh, mb, nm, pb, nh, mem;
        if (first_piece && launch) {
            row = ld_shared_s32(lrec); b = ld_shared_s32(lrec + 4); e = ld_shared_s32(lrec + 8);
            kvh = ld_shared_s32(lrec + 12); mb = ld_shared_s32(lrec + 16); nm = ld_shared_s32(lrec + 20);
            pb = ld_shared_s32(lrec + 24); nh = ld_shared_s32(lrec + 28);
            mem = lane < kDecPieceMembers ? ld_shared_s32(lrec + 32 + 4 * lane) : 0;
        } else {
            if (dealt) break;
            int taken = 0;
            if (lane == 0) taken = (int)atomicAdd(sched, 1u);
            taken = __shfl_sync(0xffffffffu, taken, 0);
            if (taken >= n_narrow) break;
            const int4* rp = reinterpret_cast<const int4*>(pieces + taken);
            const int4 x = __ldg(rp), y = __ldg(rp + 1);
            row = x.x; b = x.y; e = x.z; kvh = x.w;
            mb = y.x; nm = y.y; pb = y.z; nh = y.w;
            mem = lane < nm ? __ldg(members + mb + lane) : 0;
        }
        first_piece = false;
        int len = __ldg(seq_lens + row);
        if (e == kDecToSeqEnd) {
            // a request's trailing piece runs to its length now (within its
            // row of the table; a length below the piece's start is an error)
            if (len > ld || len < b) {
                if (lane == 0) atomicOr(err, 2u);
                len = len > ld ? (int)ld : b;
            }
            e = len;
        }
        // at least one step, so that an empty piece still writes its
        // (empty) partial rows for the merge
        for (int sp = b; sp < e || sp == b; sp += NP)
            entry(kvh, row, sp, e, sp == b ? kFirst : 0, len, pb, nh, nm, mem);
    }
    entry(-1, 0, 0, 0, 0, 0, 0, 0, 0, 0);   // the end of the stream
    cp_async_wait<0>();
    // The last lookup warp to finish restores the counter for the next call
    // (every CTA has taken its last number by then).
    if (lane == 0 && !dealt) {
        if (atomicAdd(sched + 1, 1u) + 1 == gridDim.x) {
            sched[0] = (uint32_t)f.n_init;
            sched[1] = 0u;
            __threadfence();
        }
    }
}

// The tile roles' view of wide item w.
__device__ __forceinline__ void dec_tile_info(const TcArgs& a, int w, int* info) {
    const DecItem it = a.items[w];
    int e = it.kv_end;
    const int len = __ldg(a.seq_lens + it.rep_row);
    if (e > len) {
        atomicOr(a.err, 2u);
        e = len;
    }
    info[0] = it.rep_row;
    info[1] = it.kv_begin;
    info[2] = e > it.kv_begin ? e : it.kv_begin;
    info[3] = it.kvh;
    info[4] = it.n_mem * a.G;
    info[5] = it.mem_begin;
    info[6] = it.partial_base;
}

}  // namespace
}  // namespace sgl
