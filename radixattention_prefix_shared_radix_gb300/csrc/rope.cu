// Rotary positions, and the append of new keys and values to the paged pools
// with the rotation on the way.
//
// Rotation: with angle t = p f_j for position p and pair j, each pair (a, b)
// of a head becomes (a cos t - b sin t, b cos t + a sin t), computed in fp32
// and rounded once.  Pair j is elements (j, j + rot/2) (half layout) or
// (2j, 2j + 1) (pairs layout) of the head's rotated part.
//
// Angles: a table of cosines and sines would have to be read (512 bytes per
// token of a 128-wide head, and a table as long as the longest context), and
// p f_j in fp32 is off by p 2^-24 radians, which is wrong beyond a few
// thousand positions.  Instead a frequency (f_j as a double) is a 64-bit
// fixed-point fraction of a turn: p times it, modulo 2^64, is the fraction of
// a turn that the angle stands at, off by p 2^-64 turns at most (2^-30 of a
// radian at the farthest position), with one integer product and no range
// reduction.  The nearest quarter turn is split off before the
// conversion to fp32, so that the fp32 angle is at most an eighth of a turn.
//
// Work: a warp works on one token by itself -- it finds the request, position
// and slot, puts the token's sines and cosines into its own piece of shared
// memory, and takes units of 16 elements (two 16-byte pieces that the rotation
// pairs up; 32 bytes for fp32) from the new rows to the outputs.  A token's
// heads are dealt to the two or four warps of its CTA, or to several CTAs.  The
// loads of a warp's next group of units are in flight while it works on one,
// the first ones before the position is known.
// Memory-bound: rows are read and written once, and what counts is how many
// warps have loads in flight: 36 of them per SM (56 registers) with one group
// ahead, 16384 bf16 rows of 72 heads take 91.4 us (6.6 TB/s, 0.97 of the
// measured copy); 32 warps two groups ahead 92-95, 24 warps 96-102.  8192 prompt
// tokens of 32 + 2 * 8 heads into a 4-bit pool take 33 us (26 at the copy's
// rate; 43 with lookups and tables shared by a CTA between barriers and units
// dealt thread by thread, whose bookkeeping cost more than the rotation).
// The same rows into the other pools, against their bytes at the copy's rate:
// fp32 64.0 us (59.4), bf16 33.4 (29.7), E4M3 33.8 (27.2; 16 divisions a
// unit); 8192 rows of 16 x 576 and an MLA row each 51.9 (47.3), 40.5 with the
// queries in place, whose part that is not rotated is still read; 8192 fp32
// rows of 72 heads, rotated, 94.6 (89.1).
//
// ["SGLang 深度解读" (luoboask.github.io) section "5. Attention 层": the new
// tokens' K/V are stored into token_to_kv_pool at their req_to_token slots
// before attention; CS349D lecture-16 notes §5.1: the position part of an
// MLA row is rotated, its latent part is not]

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "common.h"
#include "fp4.cuh"

// Frequencies of the rotated pairs (host object).
struct sgl_rope_table {
    sgl_rope_params p;
    double amplitude;                // multiplies cos and sin
    uint64_t turn[SGL_ROPE_MAX_DIM / 2];   // f_j 2^64 / (2 pi): fractions of a turn per position
};

namespace {

using namespace sgldev;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHalf = SGL_ROPE_MAX_DIM / 2;

enum { kPoolNone = 0, kPoolSame = 1, kPoolE4m3 = 2, kPoolFp4 = 3 };

struct RopeArgs {
    // rows [n_rows, heads, d], a row every `stride` elements
    const void *q, *k, *v;
    int64_t qs, ks, vs;
    void *qo, *ko;                   // rotated rows (ko: without pools)
    int64_t qos, kos;
    uint8_t *kp, *vp;                // pools
    const int32_t* positions;        // rotation only
    const int32_t* r2t;
    int64_t ld;
    const int32_t *lens, *ext;       // ext null: one token per request at lens[r] - 1
    uint32_t* err;
    int64_t n_rows, num_slots;
    int B, Hq, Hk, Hv, d;
    int rot, off;                    // rotated part [off, off + rot) of a head (rot 0: none)
    int pairs;                       // layout
    int lt, lg;                      // log2 of the tokens per CTA, of a power of two of units per head
    int groups, gq, gk;              // groups of 32 units of a token: in all; of q, of q and k (powers of two)
    int row_bytes;                   // bytes of a pool row
    uint32_t uph_inv;                // ceil(2^32 / units per head): exact quotients of units below 2^16
    bool copy_q;                     // q_out is not q: the part that is not rotated is copied
    float k_scale, v_scale, amp_hi, amp_lo;
    float k_six, v_six, k_sixth, v_sixth;    // 6 k_scale, 6 v_scale and their reciprocals
    uint64_t turn[kMaxHalf];
};

// request and index within it of new row n: the first r with
// ext[0] + .. + ext[r] > n.  One warp, 128 requests per round of loads.  (Rows
// and their sums stay below 2^30: at most kMaxRows rows a call, a length counts
// at most that.)
constexpr int kMaxRows = 1 << 24;
__device__ __forceinline__ bool find_request(const int32_t* ext, int B, int n, int lane, int* req, int* idx) {
    int acc = 0;
    for (int b = 0; b < B; b += 128) {
        int e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int r = b + 32 * c + lane;
            e[c] = r < B ? min(max(__ldg(ext + r), 0), kMaxRows) : 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (b + 32 * c >= B) break;
            int s = e[c];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, acc + s > n);
            if (hit) {
                const int l = __ffs(hit) - 1;
                *req = b + 32 * c + l;
                *idx = n - acc - __shfl_sync(0xffffffffu, s - e[c], l);
                return true;
            }
            acc += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    return false;
}

// cos and sin of the angle `ph` / 2^64 turns, times the amplitude (hi + lo),
// each within a little over half a unit in the last place: appended keys are
// quantised next, and a wrong last bit can move a code.  After the nearest
// quarter turn is taken off, the angle x = xh + xl (two floats) is at most
// pi / 4; sine and cosine are the Taylor sums to x^11 and x^12 (the terms left
// out are below 2^-36), ordered so that everything but one addition is small.
__device__ __forceinline__ float2 cos_sin_turn(uint64_t ph, float amp_hi, float amp_lo) {
    const uint32_t quarter = (uint32_t)((ph + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(ph - ((uint64_t)quarter << 62));     // [-1/8, 1/8) turn
    // rest = 2^8 (nh + nl) to within 2^8, nh a float of its bits from 40 on and
    // nl of the 32 below; angles below 2^-19 of a turn are taken 2^16 times as
    // large, so that nh holds the leading bits and the sum is good to 2^-30 of
    // itself, however small
    uint32_t lo = (uint32_t)rest;
    int32_t hi = (int32_t)(rest >> 32);
    const bool small = (uint32_t)(hi + (1 << 13)) < (1u << 14);
    if (small) {
        hi = (int32_t)__funnelshift_l(lo, (uint32_t)hi, 16);
        lo <<= 16;
    }
    const float nh = (float)(hi & ~0xff) * 0x1p24f;
    const float nl = (float)__funnelshift_l(lo, (uint32_t)hi, 24);
    // 2 pi 2^-56 as the sum of two floats
    constexpr double kTurn = 6.283185307179586476925286766559 * 0x1p-56;
    constexpr float kTurnH = (float)kTurn, kTurnL = (float)(kTurn - (double)kTurnH);
    const float kH = small ? kTurnH * 0x1p-16f : kTurnH, kL = small ? kTurnL * 0x1p-16f : kTurnL;
    const float xh0 = nh * kH;
    const float xl0 = fmaf(nh, kL, fmaf(nl, kH, fmaf(nh, kH, -xh0)));
    const float x = xh0 + xl0, xl = xl0 - (x - xh0);
    const float z = x * x;
    float ps = fmaf(z, -1.f / 39916800.f, 1.f / 362880.f);
    ps = fmaf(z, ps, -1.f / 5040.f);
    ps = fmaf(z, ps, 1.f / 120.f);
    ps = fmaf(z, ps, -1.f / 6.f);
    float pc = fmaf(z, 1.f / 479001600.f, -1.f / 3628800.f);
    pc = fmaf(z, pc, 1.f / 40320.f);
    pc = fmaf(z, pc, -1.f / 720.f);
    pc = fmaf(z, pc, 1.f / 24.f);
    // sin = x + (x z ps + xl cos): sh + sl; cos = 1 - z / 2 + (z^2 pc - x xl): ch + cl
    const float half = 0.5f * z, ch0 = 1.f - half;
    const float zl = fmaf(x, x, -z);                       // x^2 = z + zl
    const float st = fmaf(x * z, ps, xl * ch0);
    const float ct = ((1.f - ch0) - half) + (fmaf(z * z, pc, -x * xl) - 0.5f * zl);
    // times the amplitude, rounded once: (h + l) (amp_hi + amp_lo)
    auto times = [&](float h, float l) {
        const float t = h * amp_hi;
        return t + (fmaf(h, amp_hi, -t) + fmaf(l, amp_hi, h * amp_lo));
    };
    const float s = times(x, st), c = times(ch0, ct);
    float2 r = (quarter & 1u) ? make_float2(-s, c) : make_float2(c, s);
    if (quarter & 2u) r = make_float2(-r.x, -r.y);
    return r;
}

// eight consecutive elements as loaded
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
    uint4 w;
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        w = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(base) + at);
    }
    __device__ __forceinline__ void put(bf16* dst) const { *reinterpret_cast<uint4*>(dst) = w; }
    __device__ __forceinline__ void set(const float* x) {
        w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void put(float* dst) const {
        reinterpret_cast<float4*>(dst)[0] = a;
        reinterpret_cast<float4*>(dst)[1] = b;
    }
    __device__ __forceinline__ void set(const float* x) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
// largest magnitude of eight bf16 values as a pair of 16-bit patterns
// (patterns order like magnitudes, NaN above infinity)
__device__ __forceinline__ uint32_t amax8(uint4 w) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
}

// Exact ties are common where a bf16 value is divided by a product of few bits,
// and must round as the quotient does, so a multiplication by a reciprocal
// alone will not do.  One correction makes it the rounded quotient (Markstein
// 1990: q = z y, then q + (z - q f) y, with y the rounded reciprocal of f),
// within this range of f and for |z| < 2^60, so that no product overflows (an
// infinite q would be corrected to NaN); other operands are divided.  The
// remainder is taken as q f - z, which keeps the sign of a zero.
__device__ __forceinline__ bool quick_range(float f) { return f >= 0x1p-60f && f <= 0x1p60f; }
constexpr uint32_t kQuickTop = (127u + 60u) << 7;      // bf16 pattern of 2^60
__device__ __forceinline__ float quotient(float z, float f, float y) {
    const float q = z * y;
    return fmaf(fmaf(q, f, -z), -y, q);
}

// Code of a block's scale: the E4M3 value nearest to amax / s6, amax the
// block's largest magnitude (the larger of two bf16 patterns), s6 = 6 scale
// and y6 its rounded reciprocal.
__device__ __forceinline__ uint32_t block_scale(uint32_t m, float s6, float y6) {
    const uint32_t bits = max(m & 0xffffu, m >> 16);
    const float amax = __uint_as_float(bits << 16);
    return e4m3_of(bits < kQuickTop && quick_range(s6) ? quotient(amax, s6, y6) : __fdiv_rn(amax, s6));
}

// c = z / f for a block of bf16 values of magnitudes up to `m` (a pair of
// patterns), f >= 0; zeros where f is 0.
__device__ __forceinline__ void divide16(const float* z, float f, uint32_t m, float* c) {
    if (quick_range(f) && max(m & 0xffffu, m >> 16) < kQuickTop) {
        const float y = __frcp_rn(f);
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j] = quotient(z[j], f, y);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j] = f > 0.f ? __fdiv_rn(z[j], f) : z[j] * 0.f;
    }
}

// What a lane works on in group `id` of its token: unit c of head h of q, k or
// v (part 0, 1, 2).  PART >= 0 (a head has a power of two of units up to 32):
// a lane's c stays and a group lies within one part, which the caller knows,
// so that the part's arguments are plain constants; PART < 0: found per lane.
struct Place {
    int part, h, c;
    bool ok;
};
template <int PART>
__device__ __forceinline__ Place place(const RopeArgs& a, int id, int lane) {
    Place x;
    if constexpr (PART >= 0) {
        x.part = PART;
        id -= PART == 0 ? 0 : PART == 1 ? a.gq : a.gk;
        x.h = (id << (5 - a.lg)) + (lane >> a.lg);
        x.c = lane & ((1 << a.lg) - 1);
        x.ok = x.h < (PART == 0 ? a.Hq : PART == 1 ? a.Hk : a.Hv);
    } else {
        const int u = id * 32 + lane, uph = a.d >> 4;
        x.h = (int)__umulhi((uint32_t)u, a.uph_inv);         // u / uph
        x.c = u - x.h * uph;
        x.ok = x.h < a.Hq + a.Hk + a.Hv;
        x.part = x.h < a.Hq ? 0 : x.h < a.Hq + a.Hk ? 1 : 2;
        x.h -= x.part == 0 ? 0 : x.part == 1 ? a.Hq : a.Hq + a.Hk;
    }
    return x;
}
template <int N>
struct Part {
    static constexpr int value = N;
};

template <typename T, int POOL, bool POW2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 9 : 6) rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float cs[kWarps][2][kMaxHalf];    // cosines, sines of a warp's token
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);    // (known to be the same for the warp)
    const int64_t n = ((int64_t)blockIdx.x << a.lt) + (warp & ((1 << a.lt) - 1));
    const int step = (kWarps >> a.lt) * gridDim.y;             // warps per token
    const int id0 = (warp >> a.lt) + (kWarps >> a.lt) * blockIdx.y;
    grid_dep_wait();      // launched as a programmatic dependent: inputs may come from the kernel before
    grid_dep_launch();
    if (n >= a.n_rows || id0 >= a.groups) return;
    const int rblk = a.off >> 4, rend = rblk + (a.rot >> 4);   // rotated units of a head
    const T* const qrow = static_cast<const T*>(a.q) + n * a.qs;
    const T* const krow = static_cast<const T*>(a.k) + n * a.ks;
    const T* const vrow = static_cast<const T*>(a.v) + n * a.vs;
    T* const qout = static_cast<T*>(a.qo) + n * a.qos;
    T* const kout = static_cast<T*>(a.ko) + n * a.kos;
    auto rotated = [&](const Place& x) { return x.part < 2 && x.c >= rblk && x.c < rend; };
    // a unit's two runs of eight elements
    auto run0 = [&](const Place& x, bool rot) { return rot && !a.pairs ? a.off + 8 * (x.c - rblk) : 16 * x.c; };
    auto run1 = [&](const Place& x, bool rot) {
        return rot && !a.pairs ? a.off + 8 * (x.c - rblk) + (a.rot >> 1) : 16 * x.c + 8;
    };
    Eight<T> nx[2];       // the next group's
    auto fetch_of = [&](auto part, int id) {
        const Place x = place<decltype(part)::value>(a, id, lane);
        if (!x.ok) return;
        const T* p = (x.part == 0 ? qrow : x.part == 1 ? krow : vrow) + x.h * a.d;
        const bool rot = rotated(x);
        nx[0].load(p, run0(x, rot));
        nx[1].load(p, run1(x, rot));
    };
    // f(part, ..) for the part that group id lies in
    auto by_part = [&](int id, auto f) {
        if constexpr (!POW2)
            f(Part<-1>{});
        else if (id < a.gq)
            f(Part<0>{});
        else if (id < a.gk)
            f(Part<1>{});
        else
            f(Part<2>{});
    };
    auto fetch = [&](int id) {
        if (id < a.groups) by_part(id, [&](auto part) { fetch_of(part, id); });
    };
    fetch(id0);
    // position and slot: -1 where there is nothing to do
    int pos = -1, slot = -1;
    if constexpr (POOL == kPoolNone) {
        pos = __ldg(a.positions + n);
    } else {
        int r = (int)n, i = 0;
        if (!a.ext || find_request(a.ext, a.B, (int)n, lane, &r, &i)) {
            const int64_t p = a.ext ? (int64_t)__ldg(a.lens + r) + i : (int64_t)__ldg(a.lens + r) - 1;
            // no context (decode): nothing to append; past the table: an error
            if (p >= a.ld || (p < 0 && a.ext)) {
                if (lane == 0 && id0 == 0) atomicOr(a.err, 2u);
            } else if (p >= 0) {
                pos = (int)p;
                slot = __ldg(a.r2t + (int64_t)r * a.ld + p);
                if (slot < 0 || slot >= a.num_slots) {
                    if (lane == 0 && id0 == 0) atomicOr(a.err, 1u);
                    slot = -1;
                }
            }
        }
    }
    if (pos < 0) return;
    const int half = a.rot >> 1;
    for (int j = lane; j < half; j += 32) {
        // (an ordinary load: the lanes' indices differ, which the constant
        // cache would serve one by one)
        uint64_t turn;
        asm("ld.b64 %0, [%1];" : "=l"(turn) : "l"(&a.turn[j]));
        const float2 v = cos_sin_turn((uint64_t)(uint32_t)pos * turn, a.amp_hi, a.amp_lo);
        cs[warp][0][j] = v.x;
        cs[warp][1][j] = v.y;
    }
    __syncwarp();
    // the cosines and sines of unit c's eight pairs
    float co[8], si[8];
    auto angles = [&](int c) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 u = *reinterpret_cast<const float4*>(&cs[warp][0][8 * (c - rblk) + j]);
            const float4 w = *reinterpret_cast<const float4*>(&cs[warp][1][8 * (c - rblk) + j]);
            co[j] = u.x; co[j + 1] = u.y; co[j + 2] = u.z; co[j + 3] = u.w;
            si[j] = w.x; si[j + 1] = w.y; si[j + 2] = w.z; si[j + 3] = w.w;
        }
    };
    if constexpr (POW2) {
        const int c = lane & ((1 << a.lg) - 1);
        if (c >= rblk && c < rend) angles(c);
    }
    auto work_of = [&](auto part, Eight<T> (&w)[2], int id) {
        const Place x = place<decltype(part)::value>(a, id, lane);
        const bool rot = rotated(x);
        const int e0 = run0(x, rot), e1 = run1(x, rot);
        Eight<T> r0 = w[0], r1 = w[1];          // (what is not rotated keeps its bits)
        if (rot) {
            if constexpr (!POW2) angles(x.c);
            float y[16];
            r0.get(y);
            r1.get(y + 8);
            // (written out, so that every instantiation rounds alike)
            if (a.pairs) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = y[2 * j], q = y[2 * j + 1];
                    y[2 * j] = __fmaf_rn(p, co[j], -__fmul_rn(q, si[j]));
                    y[2 * j + 1] = __fmaf_rn(q, co[j], __fmul_rn(p, si[j]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = y[j], q = y[j + 8];
                    y[j] = __fmaf_rn(p, co[j], -__fmul_rn(q, si[j]));
                    y[j + 8] = __fmaf_rn(q, co[j], __fmul_rn(p, si[j]));
                }
            }
            r0.set(y);
            r1.set(y + 8);
        }
        if (x.part == 0 || POOL == kPoolNone) {
            if (x.ok && (rot || a.copy_q)) {
                T* dst = (x.part == 0 ? qout : kout) + x.h * a.d;
                r0.put(dst + e0);
                r1.put(dst + e1);
            }
            return;
        }
        uint8_t* row = (x.part == 1 ? a.kp : a.vp) + (int64_t)max(slot, 0) * a.row_bytes;
        [[maybe_unused]] const bool live = x.ok && slot >= 0;
        if constexpr (POOL == kPoolSame) {
            if (live) {
                T* dst = reinterpret_cast<T*>(row) + x.h * a.d;
                r0.put(dst + e0);
                r1.put(dst + e1);
            }
        } else if constexpr (POOL == kPoolE4m3) {
            // quantised pools hold codes of the rows' bf16 values, as an
            // unfused rotation would have left them
            if (live) {
                const float scale = x.part == 1 ? a.k_scale : a.v_scale;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float z[8];
                    (b ? r1 : r0).get(z);
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint16_t y;
                        const float lo = __fdiv_rn(z[2 * j], scale), hi = __fdiv_rn(z[2 * j + 1], scale);
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
                        v[j] = y;
                    }
                    *reinterpret_cast<uint2*>(row + x.h * a.d + (b ? e1 : e0)) =
                        make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
                }
            }
        } else if constexpr (POOL == kPoolFp4) {
            // One block of 16 per lane.  A unit's runs are the halves of one
            // block, or, rotated in the half layout, halves of two, whose other
            // halves the neighbouring unit's lane holds: the even unit takes
            // the first block, the odd one the second (a group is of one part:
            // the whole warp is here).
            int e = e0;
            if (decltype(part)::value == 1 && !a.pairs && a.rot > 16) {
                const bool odd = (x.c - rblk) & 1;
                uint4 give = odd ? r0.w : r1.w;
                const int other = rot ? (odd ? lane - 1 : lane + 1) : lane;
                give.x = __shfl_sync(0xffffffffu, give.x, other);
                give.y = __shfl_sync(0xffffffffu, give.y, other);
                give.z = __shfl_sync(0xffffffffu, give.z, other);
                give.w = __shfl_sync(0xffffffffu, give.w, other);
                if (rot && odd) {
                    r0.w = give;
                    e = e1 - 8;
                } else if (rot) {
                    r1.w = give;
                }
            }
            if (live) {
                const bool key = x.part == 1;
                const uint32_t m = __vmaxu2(amax8(r0.w), amax8(r1.w));
                const uint32_t sf = block_scale(m, key ? a.k_six : a.v_six, key ? a.k_sixth : a.v_sixth);
                float z[16], y[16];
                r0.get(z);
                r1.get(z + 8);
                divide16(z, e4m3_value(sf) * (key ? a.k_scale : a.v_scale), m, y);
                *reinterpret_cast<uint2*>(row + fp4_code_off(x.h, a.d) + e / 2) = make_uint2(e2m1x8_of(y), e2m1x8_of(y + 8));
                row[fp4_scale_off(x.h, key ? a.Hk : a.Hv, a.d) + e / 16] = (uint8_t)sf;
            }
        }
    };
    for (int id = id0; id < a.groups; id += step) {
        Eight<T> now[2] = {nx[0], nx[1]};
        fetch(id + step);
        by_part(id, [&](auto part) { work_of(part, now, id); });
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return SGL_OK;
    sgl::set_cuda_error(static_cast<int>(e));
    return SGL_ERR_CUDA;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// rows of `heads` heads, `stride` elements apart, of es bytes each
bool rows_ok(const void* p, int64_t stride, int heads, int d, int es) {
    return p && aligned16(p) && stride >= (int64_t)heads * d && stride * es % 16 == 0;
}

template <typename T, int POOL, bool POW2>
int launch_as(RopeArgs& a, cudaStream_t s) {
    // Two tokens share a CTA (two warps each) once every SM has one; below one
    // token per SM a token's groups are spread over several CTAs.  Measured
    // with 1, 2 and 4 tokens per CTA: 8192 rows into a 4-bit pool 36.8, 32.9
    // and 34.2 us, 16384 rows of 72 heads 91.7, 91.4 and 95.6.
    constexpr int kSms = 152;
    const int heads = a.Hq + a.Hk + a.Hv, uph = a.d / 16;
    if ((int64_t)heads * uph > 0xffff - 32) return SGL_ERR_UNSUPPORTED;     // (unit numbers and their quotients)
    a.lt = a.n_rows >= 2 * kSms ? 1 : 0;
    a.uph_inv = uph > 1 ? (uint32_t)(((1ull << 32) + uph - 1) / uph) : 0u;
    a.lg = 0;
    while ((1 << a.lg) < uph) ++a.lg;
    const int per = std::max(1, 32 / uph);                                  // heads per group
    if (POW2) {
        a.gq = (a.Hq + per - 1) / per;
        a.gk = a.gq + (a.Hk + per - 1) / per;
        a.groups = a.gk + (a.Hv + per - 1) / per;
    } else {
        a.groups = (heads * uph + 31) / 32;
    }
    int slices = 1;
    if (a.n_rows < kSms)
        slices = (int)std::min<int64_t>((kSms + a.n_rows - 1) / a.n_rows, (a.groups + kWarps - 1) / kWarps);
    const int64_t ctas = (a.n_rows + (1 << a.lt) - 1) >> a.lt;
    if (ctas > INT32_MAX) return SGL_ERR_UNSUPPORTED;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)slices);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, rope_kernel<T, POOL, POW2>, a));
}

template <typename T, int POOL>
int launch(RopeArgs& a, cudaStream_t s) {
    if (a.n_rows == 0 || a.Hq + a.Hk + a.Hv == 0) return SGL_OK;
    if ((a.d & (a.d - 1)) == 0 && a.d <= 512) return launch_as<T, POOL, true>(a, s);
    // other widths: rotation alone and MLA rows (the pools' heads are 64 or 128 wide)
    if constexpr (POOL == kPoolNone || (POOL == kPoolSame && sizeof(T) == 2)) return launch_as<T, POOL, false>(a, s);
    return SGL_ERR_UNSUPPORTED;
}

void set_table(RopeArgs& a, const sgl_rope_table* t) {
    if (!t) return;
    a.rot = t->p.rot_dim;
    a.off = t->p.rot_offset;
    a.pairs = t->p.layout == SGL_ROPE_PAIRS;
    a.amp_hi = (float)t->amplitude;
    a.amp_lo = (float)(t->amplitude - (double)a.amp_hi);
    std::memcpy(a.turn, t->turn, sizeof(uint64_t) * (size_t)(t->p.rot_dim / 2));
}

// 2^64 f / (2 pi) as a whole number, within one: f times 1 / (2 pi) as the sum
// of two doubles (a quotient in doubles is off by 2^-53 of itself, which the
// position multiplies: a millionth of a radian at positions near 2^31).  f <= 1
// radian, so the fraction of a turn is below 1/6.
uint64_t turn_of(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double p = f * kHi, e = std::fma(f, kHi, -p) + f * kLo;
    const double whole = std::floor(std::ldexp(p, 64));
    return (uint64_t)whole + (uint64_t)(int64_t)std::nearbyint((std::ldexp(p, 64) - whole) + std::ldexp(e, 64));
}

// the arguments that both appends share, checked
int append_rows(RopeArgs& a, const sgl_rope_table* rope, int es, int64_t n_rows, const int32_t* req_to_token, int64_t ld,
                const int32_t* lens, const int32_t* extend_lens, int32_t batch, const void* q, int64_t q_stride,
                void* q_out, int64_t q_out_stride, int Hq, int d, void* workspace, size_t ws_bytes) {
    if (n_rows < 0 || ld < 0 || (rope && rope->p.head_dim != d)) return SGL_ERR_INVALID_ARG;
    if (!extend_lens && n_rows > batch) return SGL_ERR_INVALID_ARG;
    if (n_rows > kMaxRows) return SGL_ERR_UNSUPPORTED;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % sgl::kWsAlign) != 0 || ws_bytes < sgl::kWsAlign)
        return SGL_ERR_WORKSPACE;
    if (n_rows > 0 && (!req_to_token || !lens)) return SGL_ERR_INVALID_ARG;
    if (!q != !q_out) return SGL_ERR_INVALID_ARG;
    if (n_rows > 0 && q && !(rows_ok(q, q_stride, Hq, d, es) && rows_ok(q_out, q_out_stride, Hq, d, es)))
        return SGL_ERR_INVALID_ARG;
    if (q && q == q_out && q_stride != q_out_stride) return SGL_ERR_INVALID_ARG;
    set_table(a, rope);
    a.q = q;
    a.qs = q_stride;
    a.qo = q_out;
    a.qos = q_out_stride;
    a.Hq = q ? Hq : 0;
    a.copy_q = q != q_out;
    a.r2t = req_to_token;
    a.ld = ld;
    a.lens = lens;
    a.ext = extend_lens;
    a.B = batch;
    a.err = static_cast<uint32_t*>(workspace);
    a.n_rows = n_rows;
    a.d = d;
    return SGL_OK;
}

}  // namespace

namespace sgl {
int check_params(const sgl_attn_params* p);
}

extern "C" {

int sgl_fp4_row_bytes(int32_t num_kv_heads, int32_t head_dim, int64_t* bytes) {
    if (!bytes || num_kv_heads <= 0) return SGL_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || num_kv_heads > (1 << 16)) return SGL_ERR_UNSUPPORTED;
    *bytes = fp4_row_bytes(num_kv_heads, head_dim);
    return SGL_OK;
}

int sgl_rope_create(const sgl_rope_params* p, sgl_rope_table** out) {
    if (!p || !out) return SGL_ERR_INVALID_ARG;
    const int n = p->rot_dim;
    if (p->head_dim <= 0 || n <= 0 || p->rot_offset < 0 || (int64_t)p->rot_offset + n > p->head_dim)
        return SGL_ERR_INVALID_ARG;
    if (!(p->theta > 1.0) || !std::isfinite(p->theta)) return SGL_ERR_INVALID_ARG;
    if (!(p->attention_factor >= 0.0) || !std::isfinite((float)p->attention_factor)) return SGL_ERR_INVALID_ARG;
    if (p->layout != SGL_ROPE_HALF && p->layout != SGL_ROPE_PAIRS) return SGL_ERR_UNSUPPORTED;
    if (p->head_dim % 16 || p->head_dim > 1024 || n % 16 || n > SGL_ROPE_MAX_DIM || p->rot_offset % 16)
        return SGL_ERR_UNSUPPORTED;
    if (p->layout == SGL_ROPE_HALF && n != 16 && n % 32) return SGL_ERR_UNSUPPORTED;
    const int kind = p->scaling;
    if (kind < SGL_ROPE_SCALE_NONE || kind > SGL_ROPE_SCALE_BANDED) return SGL_ERR_UNSUPPORTED;
    const double by = p->factor;
    if (kind != SGL_ROPE_SCALE_NONE && !(by >= 1.0 && std::isfinite(by))) return SGL_ERR_INVALID_ARG;
    const bool bands = kind == SGL_ROPE_SCALE_YARN || kind == SGL_ROPE_SCALE_BANDED;
    if (bands && !(p->original_positions > 0 && p->low > 0.0 && p->high > p->low && std::isfinite(p->high)))
        return SGL_ERR_INVALID_ARG;
    auto* t = new (std::nothrow) sgl_rope_table();
    if (!t) return SGL_ERR_INVALID_ARG;
    t->p = *p;
    const double two_pi = 6.283185307179586476925286766559;
    const double orig = (double)p->original_positions;
    double theta = p->theta;
    if (kind == SGL_ROPE_SCALE_NTK) theta *= std::pow(by, (double)n / (n - 2));
    double lo = 0.0, hi = 1.0;
    if (kind == SGL_ROPE_SCALE_YARN) {
        // the pair index at which a pair makes `turns` turns over the original positions
        auto index = [&](double turns) { return n * std::log(orig / (turns * two_pi)) / (2.0 * std::log(p->theta)); };
        lo = std::fmax(std::floor(index(p->high)), 0.0);
        hi = std::fmin(std::ceil(index(p->low)), n - 1.0);
        if (hi <= lo) hi = lo + 0.001;
    }
    for (int j = 0; j < n / 2; ++j) {
        double f = std::pow(theta, -2.0 * j / n);
        if (kind == SGL_ROPE_SCALE_LINEAR) {
            f /= by;
        } else if (kind == SGL_ROPE_SCALE_YARN) {
            const double w = std::fmin(std::fmax((j - lo) / (hi - lo), 0.0), 1.0);
            f = f / by * w + f * (1.0 - w);
        } else if (kind == SGL_ROPE_SCALE_BANDED) {
            const double w = std::fmin(std::fmax((orig * f / two_pi - p->low) / (p->high - p->low), 0.0), 1.0);
            f = f / by * (1.0 - w) + f * w;
        }
        t->turn[j] = turn_of(f);
    }
    double amp = p->attention_factor;
    if (amp == 0.0) amp = kind == SGL_ROPE_SCALE_YARN ? 0.1 * std::log(by) + 1.0 : 1.0;
    t->amplitude = amp;
    *out = t;
    return SGL_OK;
}

void sgl_rope_destroy(sgl_rope_table* t) { delete t; }

int sgl_rope(const sgl_rope_table* rope, int32_t dtype, const void* q, int64_t q_stride, int32_t num_q_heads,
             const void* k, int64_t k_stride, int32_t num_k_heads, const int32_t* positions, int64_t n_rows, void* q_out,
             int64_t q_out_stride, void* k_out, int64_t k_out_stride, sgl_stream_t stream) {
    if (!rope || n_rows < 0 || num_q_heads < 0 || num_k_heads < 0) return SGL_ERR_INVALID_ARG;
    if (dtype != SGL_DTYPE_F32 && dtype != SGL_DTYPE_BF16) return SGL_ERR_UNSUPPORTED;
    if (n_rows == 0) return SGL_OK;
    const int d = rope->p.head_dim, es = dtype == SGL_DTYPE_F32 ? 4 : 2;
    if ((int64_t)num_q_heads + num_k_heads > INT32_MAX / 1024) return SGL_ERR_UNSUPPORTED;
    if (!positions) return SGL_ERR_INVALID_ARG;
    if (num_q_heads > 0 && !(rows_ok(q, q_stride, num_q_heads, d, es) && rows_ok(q_out, q_out_stride, num_q_heads, d, es)))
        return SGL_ERR_INVALID_ARG;
    if (num_k_heads > 0 && !(rows_ok(k, k_stride, num_k_heads, d, es) && rows_ok(k_out, k_out_stride, num_k_heads, d, es)))
        return SGL_ERR_INVALID_ARG;
    // in place: the same rows
    if (num_q_heads > 0 && q == q_out && q_stride != q_out_stride) return SGL_ERR_INVALID_ARG;
    if (num_k_heads > 0 && k == k_out && k_stride != k_out_stride) return SGL_ERR_INVALID_ARG;
    RopeArgs a{};
    set_table(a, rope);
    a.q = q;
    a.k = k;
    a.qs = q_stride;
    a.ks = k_stride;
    a.qo = q_out;
    a.ko = k_out;
    a.qos = q_out_stride;
    a.kos = k_out_stride;
    a.positions = positions;
    a.n_rows = n_rows;
    a.Hq = num_q_heads;
    a.Hk = num_k_heads;
    a.d = d;
    a.copy_q = (num_q_heads > 0 && q != q_out) || (num_k_heads > 0 && k != k_out);
    auto s = reinterpret_cast<cudaStream_t>(stream);
    return es == 4 ? launch<float, kPoolNone>(a, s) : launch<bf16, kPoolNone>(a, s);
}

int sgl_kv_append(const sgl_rope_table* rope, const sgl_attn_params* params, const void* q, int64_t q_stride,
                  const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, void* k_pool, void* v_pool,
                  const int32_t* req_to_token, int64_t ld, const int32_t* lens, const int32_t* extend_lens,
                  int64_t n_rows, void* q_out, int64_t q_out_stride, void* workspace, size_t ws_bytes,
                  sgl_stream_t stream) {
    const int st = sgl::check_params(params);
    if (st) return st;
    const int d = params->head_dim, Hkv = params->num_kv_heads, es = params->dtype == SGL_DTYPE_F32 ? 4 : 2;
    if ((int64_t)params->num_qo_heads + 2 * (int64_t)Hkv > INT32_MAX / 1024) return SGL_ERR_UNSUPPORTED;
    RopeArgs a{};
    if (const int e = append_rows(a, rope, es, n_rows, req_to_token, ld, lens, extend_lens, params->batch, q, q_stride,
                                  q_out, q_out_stride, params->num_qo_heads, d, workspace, ws_bytes))
        return e;
    if (n_rows == 0) return SGL_OK;
    if (!rows_ok(k_new, k_stride, Hkv, d, es) || !rows_ok(v_new, v_stride, Hkv, d, es)) return SGL_ERR_INVALID_ARG;
    if (!k_pool || !v_pool || !aligned16(k_pool) || !aligned16(v_pool)) return SGL_ERR_INVALID_ARG;
    a.k = k_new;
    a.v = v_new;
    a.ks = k_stride;
    a.vs = v_stride;
    a.kp = static_cast<uint8_t*>(k_pool);
    a.vp = static_cast<uint8_t*>(v_pool);
    a.num_slots = params->num_slots;
    a.Hk = a.Hv = Hkv;
    a.k_scale = params->k_scale;
    a.v_scale = params->v_scale;
    a.k_six = 6.f * a.k_scale;
    a.v_six = 6.f * a.v_scale;
    a.k_sixth = 1.f / a.k_six;
    a.v_sixth = 1.f / a.v_six;
    auto s = reinterpret_cast<cudaStream_t>(stream);
    switch (params->dtype) {
        case SGL_DTYPE_F32: a.row_bytes = Hkv * d * 4; return launch<float, kPoolSame>(a, s);
        case SGL_DTYPE_BF16: a.row_bytes = Hkv * d * 2; return launch<bf16, kPoolSame>(a, s);
        case SGL_DTYPE_BF16_FP8KV: a.row_bytes = Hkv * d; return launch<bf16, kPoolE4m3>(a, s);
        default: a.row_bytes = fp4_row_bytes(Hkv, d); return launch<bf16, kPoolFp4>(a, s);
    }
}

int sgl_mla_kv_append(const sgl_rope_table* rope, const sgl_mla_params* params, const void* q, int64_t q_stride,
                      const void* kv_new, int64_t kv_stride, void* kv_pool, const int32_t* req_to_token, int64_t ld,
                      const int32_t* lens, const int32_t* extend_lens, int64_t n_rows, void* q_out,
                      int64_t q_out_stride, void* workspace, size_t ws_bytes, sgl_stream_t stream) {
    if (!params || params->batch < 0 || params->num_slots < 0 || params->page_size < 1) return SGL_ERR_INVALID_ARG;
    const int H = params->num_qo_heads, d = 576;
    if (params->latent_dim != 512 || params->rope_dim != 64 || (H != 16 && H != 32 && H != 64 && H != 128) ||
        params->num_slots > INT32_MAX)
        return SGL_ERR_UNSUPPORTED;
    RopeArgs a{};
    if (const int e = append_rows(a, rope, 2, n_rows, req_to_token, ld, lens, extend_lens, params->batch, q, q_stride,
                                  q_out, q_out_stride, H, d, workspace, ws_bytes))
        return e;
    if (n_rows == 0) return SGL_OK;
    if (!rows_ok(kv_new, kv_stride, 1, d, 2) || !kv_pool || !aligned16(kv_pool)) return SGL_ERR_INVALID_ARG;
    a.k = kv_new;
    a.ks = kv_stride;
    a.kp = static_cast<uint8_t*>(kv_pool);
    a.num_slots = params->num_slots;
    a.Hk = 1;
    a.Hv = 0;
    a.row_bytes = d * 2;
    return launch<bf16, kPoolSame>(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
