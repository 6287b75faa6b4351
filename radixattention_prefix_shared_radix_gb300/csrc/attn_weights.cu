// The attention weights that cached tokens get from a call's queries, summed
// over query rows and heads, added to the scores that the tokens have gathered.
//
// With s = sm_scale <q, k_p> and the row's log-sum-exp L from the attention
// call, a weight is exp(s - L): no second softmax, one product Q K^T and one
// exponential per (row, head, position), and a sum over rows.

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "common.h"
#include "weights.cuh"

namespace {

using namespace sgldev;
using namespace sgl::wts;
namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Chunks over fp32 pools, on CUDA cores (exact products): a cluster of CTAs per
// (tile of 64 positions, request) deals the KV heads among its CTAs and adds
// their sums through distributed shared memory, in order.  A CTA takes 64 rows at
// a time; a thread multiplies four positions by four rows, so that eight 16-byte
// reads of shared memory, which bound it, feed 64 multiply-adds (4 x 40 to 96
// tokens of 32 heads behind 500 to 2000 139 us, 26 TFLOP/s; 2 x 1000 tokens of 64
// heads behind up to 500 1.44 ms, 17 TFLOP/s; one position by four rows took three
// times as long).
// ---------------------------------------------------------------------------
constexpr int kF32Cluster = 8, kF32Tile = 64;
template <int D>
constexpr int f32_smem() {
    return 2 * kF32Tile * (D + 4) * 4;
}

template <int D>
__global__ void __launch_bounds__(256) weights_chunk_f32(const __grid_constant__ WeightArgs a) {
    constexpr int RS = D + 4, T = kF32Tile;
    extern __shared__ __align__(16) float sk[];          // T keys, then T query rows
    float* const sq = sk + T * RS;
    __shared__ float sl[T], sums[T];
    __shared__ int32_t slots[T];
    __shared__ int64_t before_s;
    cg::cluster_group cl = cg::this_cluster();
    const int r = blockIdx.y, tid = threadIdx.x, t0 = blockIdx.x * T;
    const int C = gridDim.z, part = blockIdx.z;          // (the cluster lies along z)
    grid_dep_wait();
    grid_dep_launch();
    if (tid < 32) {
        int64_t s = 0;
        for (int b = tid; b < r; b += 32) s += max(__ldg(a.ext + b), 0);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) before_s = s;
    }
    __syncthreads();
    const int len = __ldg(a.lens + r), ext = __ldg(a.ext + r);
    const Asked x = asked(a, len, ext, before_s);
    // (lengths that the tables do not hold, or longer than the host's longest: its scores stay as they were)
    if ((x.total == 0 && (len | ext) != 0) || x.total > (int)gridDim.x * T) {
        if (tid == 0 && t0 == 0) atomicOr(a.err, 2u);
        return;
    }
    if (t0 >= x.total) return;                           // (the whole cluster)
    if (tid < T) {
        int32_t slot = -1;
        if (t0 + tid < x.total) {
            slot = __ldg(a.r2t + r * a.ld + t0 + tid);
            if (slot < 0 || slot >= a.num_slots) {
                atomicOr(a.err, 1u);
                slot = -1;
            }
        }
        slots[tid] = slot;
    }
    const int py = tid >> 4, rx = tid & 15;              // positions py + 16 i, rows rx + 16 j
    // (the sums of eight blocks, 32 weights, are added with what each addition
    // rounds off kept: a position's rows may be many thousand blocks)
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, off[4] = {0.f, 0.f, 0.f, 0.f}, now[4] = {0.f, 0.f, 0.f, 0.f};
    const int lg = 31 - __clz(a.G);
    const int rows = x.ask << lg;
    // (rows before the one that first sees the tile are passed over)
    const int row0 = max(t0 - x.p0, 0) << lg & ~(T - 1);
    for (int h = part; h < a.Hkv; h += C) {
        __syncthreads();
        for (int i = tid; i < T * (D / 4); i += 256) {
            const int p = i / (D / 4), c = i - p * (D / 4), slot = slots[p];
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot >= 0) v = reinterpret_cast<const float4*>(a.kp + (int64_t)slot * a.row_bytes)[h * (D / 4) + c];
            *reinterpret_cast<float4*>(&sk[p * RS + 4 * c]) = v;
        }
        for (int b = row0; b < rows; b += T) {
            __syncthreads();
            for (int i = tid; i < T * (D / 4); i += 256) {
                const int y = i / (D / 4), c = i - y * (D / 4), row = b + y;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row < rows)
                    v = reinterpret_cast<const float4*>(a.q)[((x.row + (row >> lg)) * a.Hq + (h << lg) + (row & (a.G - 1))) * (D / 4) + c];
                *reinterpret_cast<float4*>(&sq[y * RS + 4 * c]) = v;
            }
            if (tid < T) {
                const int row = b + tid;
                sl[tid] = row < rows ? a.lse[(x.row + (row >> lg)) * a.Hq + (h << lg) + (row & (a.G - 1))] : -INFINITY;
            }
            __syncthreads();
            float dot[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) dot[i][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 k[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    k[i] = *reinterpret_cast<const float4*>(&sk[(py + 16 * i) * RS + c]);
                    y[i] = *reinterpret_cast<const float4*>(&sq[(rx + 16 * i) * RS + c]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dot[i][j] = fmaf(k[i].x, y[j].x, fmaf(k[i].y, y[j].y, fmaf(k[i].z, y[j].z, fmaf(k[i].w, y[j].w, dot[i][j]))));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = b + rx + 16 * j, last = x.p0 + (row >> lg);        // (a row sees positions up to its own)
                const float l = sl[rx + 16 * j];         // (-infinity: no row, or one that adds nothing)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (l != -INFINITY && t0 + py + 16 * i <= last) now[i] += weight_of(dot[i][j], a.scale, -l);
            }
            if ((b & (7 * T)) == 7 * T || b + T >= rows) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = sum[i] + now[i], y = s - sum[i];
                    off[i] += (sum[i] - (s - y)) + (now[i] - y);
                    sum[i] = s;
                    now[i] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (off[i] == off[i]) sum[i] += off[i];          // (an infinite sum stays one)
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        if (rx == 0) sums[py + 16 * i] = sum[i];
    }
    if (C > 1)
        cl.sync();
    else
        __syncthreads();
    const int pos = t0 + tid;
    if (part == 0 && tid < T && pos < x.total) {
        float s = sums[tid];
        for (int c = 1; c < C; ++c) s += cl.map_shared_rank(sums, c)[tid];
        if (slots[tid] < 0) s = 0.f;
        const int64_t at = r * a.scores_ld + pos;
        a.out[at] = a.in && pos < x.fresh ? fmaf(a.decay, a.in[at], s) : s;
    }
    if (C > 1) cl.sync();
}

// ---------------------------------------------------------------------------
// Decode: the keys are streamed once, straight into the fragments of a matrix
// instruction.  A warp takes one KV head of 8 NR positions at a time: lane
// 4 g + t holds, of each row 8 n + g, every fourth 16-byte piece from piece t
// on.  A dot product does not ask in which order its terms come, so these
// pieces are the A operand of m16n8k16 as they are (words 2 j and 2 j + 1 of a
// piece are an instruction's two k pairs), with the query's pieces of the same
// places as B.  No shared memory and no ldmatrix lie between HBM and the
// multiplier; FP8 and 4-bit pieces become f16 on the way (exact).  fp32 keys are
// multiplied on CUDA cores, the query from shared memory.
//
// A tile of positions is shared by the CTA's warps, one per KV head (heads
// beyond eight in turns), or, with fewer heads, several per head over
// neighbouring positions; their sums meet in shared memory and are added in the
// heads' order.  Each CTA takes an equal, contiguous run of the batch's tiles, so
// a request's query stays in registers over its tiles.
// Memory-bound; what counts is the bytes in flight, loads of the next unit being
// issued before the exponentials of this one.  64 contexts of 1 to 8192 tokens, 8
// heads of 128: bf16 91.5 us (6.1 TB/s, 0.90 of the measured copy; ncu: 558 of 559
// MB read, issue slots 48%), 30 such over fp32 88.7 (5.6 TB/s).  E4M3 55.2 us (5.1
// TB/s; ncu: DRAM 56%, issue slots 38%) and 4 bits 51.7 (3.1; DRAM 35%, issue slots
// 50%) have no unit full: 16 warps an SM, each with one unit's loads ahead, wait for
// those (E4M3 30% of their cycles, 4 bits 20%), for each other and for their own
// chains.  One context of 180 tokens 4.1 us.
// Before, a CTA per 32 positions with keys and queries staged through shared
// memory took 2041 us on the bf16 batch.
// ---------------------------------------------------------------------------
template <int D, int KV>
struct Stream {
    static constexpr int RW = D * (KV == kKvF32 ? 32 : KV == 0 ? 16 : KV == 1 ? 8 : 4) / 8 / 16;   // a lane's words of a row
    static constexpr int NR = KV == kKvF32 ? 2 : KV == 2 ? 8 : 32 / RW;                        // rows of a lane
    static constexpr int PU = 8 * NR;                                                               // positions of a warp
    // CTAs of an SM: three where 80 registers do (bf16: three 92 us, two 102, on 64
    // contexts of 1 to 8192 tokens), two where they spill (E4M3 58 instead of 67,
    // 4 bits 55 instead of 97)
    static constexpr int CTAS = KV == 0 || (KV == kKvF32 && D == 64) ? 3 : 2;
};
constexpr int kStreamThreads = 256;

// 16 (8) bytes that are read once
__device__ __forceinline__ uint4 ldg_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg_once8(const void* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// D[16x8] += A[16x16] * B[16x8], f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma16816_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int KV>
__global__ void __launch_bounds__(kStreamThreads, Stream<D, KV>::CTAS) weights_decode(const __grid_constant__ WeightArgs a, int hw, int nsub) {
    using U = Stream<D, KV>;
    constexpr int NR = U::NR, RW = U::RW, PU = U::PU;
    constexpr bool F32 = KV == kKvF32;
    constexpr int QW = D / 8;                        // a lane's words of the query (16 bits)
    __shared__ float sums[2][8 * PU];                // [head warp][position of the tile]
    __shared__ __align__(16) float sq[F32 ? 8 * 8 * D : 4];
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int wh = warp % hw, sub = warp / hw, TP = PU * nsub;
    grid_dep_wait();
    grid_dep_launch();
    // this CTA's tiles [at, end) of all requests', in order
    auto tiles_of = [&](int len) { return len > 0 && len <= a.lim ? (len + TP - 1) / TP : 0; };
    int64_t total = 0;
    for (int b = lane; b < a.B; b += 32) {
        const int len = __ldg(a.lens + b);
        if ((len < 0 || len > a.lim) && blockIdx.x == 0 && warp == 0) atomicOr(a.err, 2u);
        total += tiles_of(len);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    int64_t at = total * blockIdx.x / gridDim.x;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    if (at >= end) return;
    int r = 0, tile = 0, len = 0;                    // request, tile of it, its length
    {
        int64_t acc = 0;
        for (int b = 0; b < a.B; b += 32) {
            const int l = b + lane < a.B ? __ldg(a.lens + b + lane) : 0, n = tiles_of(l);
            int s = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, acc + s > at);
            if (hit) {
                const int w = __ffs(hit) - 1;
                r = b + w;
                tile = (int)(at - acc) - __shfl_sync(0xffffffffu, s - n, w);
                len = __shfl_sync(0xffffffffu, l, w);
                break;
            }
            acc += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    auto next_tile = [&](int& r2, int& tile2, int& len2) {
        if (++tile2 >= tiles_of(len2)) {
            tile2 = 0;
            do len2 = __ldg(a.lens + ++r2);
            while (tiles_of(len2) == 0);             // (there is a next one: the caller counts)
        }
    };
    int slot[NR];
    auto load_slots = [&](int r2, int tile2, int len2) {
        const int32_t* row = a.r2t + (int64_t)r2 * a.ld;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int p = tile2 * TP + sub * PU + 8 * n + g;
            slot[n] = p < len2 ? __ldg(row + p) : -1;
        }
    };
    uint32_t raw[NR][RW], scale[KV == 2 ? NR : 1];
    uint32_t live = 0;                               // rows of the lane that a slot in the pool holds
    auto load_keys = [&](int h, int tile2, int len2) {
        live = 0;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const bool ok = slot[n] >= 0 && slot[n] < a.num_slots;
            if (ok)
                live |= 1u << n;
            else if (tile2 * TP + sub * PU + 8 * n + g < len2)
                atomicOr(a.err, 1u);
            const uint8_t* row = a.kp + (int64_t)(ok ? slot[n] : 0) * a.row_bytes;
            if constexpr (KV == 2) {
                const uint8_t* codes = row + fp4_code_off(h, D);
                const uint8_t* sf = row + fp4_scale_off(h, a.Hkv, D);
                if constexpr (D == 128) {
                    const uint4 v = ok ? ldg_once(codes + 16 * t) : make_uint4(0, 0, 0, 0);
                    raw[n][0] = v.x; raw[n][1] = v.y; raw[n][2] = v.z; raw[n][3] = v.w;
                    scale[n] = ok ? *reinterpret_cast<const uint16_t*>(sf + 2 * t) : 0;
                } else {
                    const uint2 v = ok ? ldg_once8(codes + 8 * t) : make_uint2(0, 0);
                    raw[n][0] = v.x; raw[n][1] = v.y;
                    scale[n] = ok ? sf[t] : 0;
                }
            } else {
                const uint8_t* piece = row + h * (RW * 16) + 16 * t;
#pragma unroll
                for (int i = 0; i < RW / 4; ++i) {
                    const uint4 v = ok ? ldg_once(piece + 64 * i) : make_uint4(0, 0, 0, 0);
                    raw[n][4 * i] = v.x; raw[n][4 * i + 1] = v.y; raw[n][4 * i + 2] = v.z; raw[n][4 * i + 3] = v.w;
                }
            }
        }
    };
    // the query rows of KV head h: B fragments (row g of eight) of the same
    // pieces that the keys come in, and minus the log-sum-exps of columns 2 t, 2 t + 1
    uint32_t qf[F32 ? 1 : QW];
    float l0, l1;                                    // (infinity: no row, or one that adds nothing)
    auto load_query = [&](int r2, int h) {
        const int64_t row = (int64_t)r2 * a.Hq + h * a.G;
        if constexpr (F32) {
            __syncwarp();
            for (int i = lane; i < a.G * (D / 4); i += 32)
                reinterpret_cast<float4*>(&sq[warp * 8 * D])[i] = __ldg(reinterpret_cast<const float4*>(a.q) + row * (D / 4) + i);
            __syncwarp();
            l0 = t < a.G ? -__ldg(a.lse + row + t) : INFINITY;
            l1 = t + 4 < a.G ? -__ldg(a.lse + row + t + 4) : INFINITY;
        } else {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.q) + (row + min(g, a.G - 1)) * D);
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < QW / 4; ++i) {
                // bf16: piece 4 i + t; codes: a key piece's 16 or 32 elements are consecutive ones
                const uint4 v = __ldg(q + (KV == 0 ? 4 * i + t : KV == 1 ? 8 * (i >> 1) + 2 * t + (i & 1) : (QW / 4) * t + i));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) qf[4 * i + j] = KV == 0 ? w[j] : bf16x2_to_f16x2_chk(w[j], bad);
            }
            if (bad && g < a.G && __ldg(a.lse + row + g) != -INFINITY) atomicOr(a.err, kErrQRange);
            l0 = 2 * t < a.G ? -__ldg(a.lse + row + 2 * t) : INFINITY;
            l1 = 2 * t + 1 < a.G ? -__ldg(a.lse + row + 2 * t + 1) : INFINITY;
        }
    };
    load_slots(r, tile, len);
    load_keys(wh, tile, len);
    int q_r = -1, q_h = -1;
    for (int buf = 0; at < end; ++at, buf ^= 1) {
        const int p0 = tile * TP;
        float old = 0.f;
        const int64_t score0 = (int64_t)r * a.scores_ld + p0;
        // (all but the newest token had a score)
        if (a.in && tid < TP && p0 + tid < len - 1) old = a.in[score0 + tid];
        int r2 = r, tile2 = tile, len2 = len;
        if (at + 1 < end) next_tile(r2, tile2, len2);
        float sum[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) sum[n] = 0.f;
        for (int h = wh; h < a.Hkv; h += hw) {
            const bool last = h + hw >= a.Hkv;
            if (last && at + 1 < end) load_slots(r2, tile2, len2);
            if (q_r != r || q_h != h) load_query(r, h);
            q_r = r;
            q_h = h;
            const uint32_t now = live;
            float c[F32 ? NR * 2 : NR / 2][4];
            if constexpr (F32) {
                // (lane t keeps the products of query rows t and t + 4)
#pragma unroll
                for (int n = 0; n < NR; ++n) c[n][0] = c[n][1] = 0.f;
                for (int j = 0; j < a.G; ++j) {
                    const float4* q = reinterpret_cast<const float4*>(&sq[(warp * 8 + j) * D]);
                    float dot[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) dot[n] = 0.f;
#pragma unroll
                    for (int i = 0; i < RW / 4; ++i) {
                        const float4 y = q[4 * i + t];
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            dot[n] = fmaf(__uint_as_float(raw[n][4 * i]), y.x, dot[n]);
                            dot[n] = fmaf(__uint_as_float(raw[n][4 * i + 1]), y.y, dot[n]);
                            dot[n] = fmaf(__uint_as_float(raw[n][4 * i + 2]), y.z, dot[n]);
                            dot[n] = fmaf(__uint_as_float(raw[n][4 * i + 3]), y.w, dot[n]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const float all = quad_sum(dot[n]);
                        if (j == t) c[n][0] = all;
                        if (j == t + 4) c[n][1] = all;
                    }
                }
            } else {
#pragma unroll
                for (int m = 0; m < NR / 2; ++m) {
                    c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
                    const uint32_t* x = raw[2 * m];
                    const uint32_t* y = raw[2 * m + 1];
                    if constexpr (KV == 0) {
#pragma unroll
                        for (int i = 0; i < RW; i += 2) {
                            const uint32_t f[4] = {x[i], y[i], x[i + 1], y[i + 1]};
                            mma16816(c[m], f, qf[i], qf[i + 1]);
                        }
                    } else if constexpr (KV == 1) {
#pragma unroll
                        for (int i = 0; i < RW; ++i) {
                            uint32_t x0, x1, y0, y1;
                            e4m3x4_to_f16(x[i], x0, x1);
                            e4m3x4_to_f16(y[i], y0, y1);
                            mma16816_f16(c[m], x0, y0, x1, y1, qf[2 * i], qf[2 * i + 1]);
                        }
                    } else {
                        const uint32_t xs = e4m3x2_to_f16(scale[2 * m]), ys = e4m3x2_to_f16(scale[2 * m + 1]);
#pragma unroll
                        for (int i = 0; i < RW; ++i) {
                            // (a word is half a block of 16)
                            const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
                            const uint32_t xf = __byte_perm(xs, 0, sel), yf = __byte_perm(ys, 0, sel);
                            uint32_t u[4], w[4];
                            e2m1x8_to_f16(x[i], u);
                            e2m1x8_to_f16(y[i], w);
#pragma unroll
                            for (int j = 0; j < 4; j += 2)
                                mma16816_f16(c[m], hmul2_u(u[j], xf), hmul2_u(w[j], yf), hmul2_u(u[j + 1], xf),
                                             hmul2_u(w[j + 1], yf), qf[4 * i + j], qf[4 * i + j + 1]);
                        }
                    }
                }
            }
            // the next keys are on their way while this unit is finished
            if (!last)
                load_keys(h + hw, tile, len);
            else if (at + 1 < end)
                load_keys(wh, tile2, len2);
            // (columns that add nothing may hold infinities and NaN)
            const bool v0 = l0 != INFINITY, v1 = l1 != INFINITY;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float x0 = F32 ? c[n][0] : c[n / 2][2 * (n & 1)], x1 = F32 ? c[n][1] : c[n / 2][2 * (n & 1) + 1];
                const float w0 = weight_of(x0, a.scale, l0), w1 = weight_of(x1, a.scale, l1);
                if (now >> n & 1u) sum[n] += (v0 ? w0 : 0.f) + (v1 ? w1 : 0.f);
            }
        }
        float* const out = sums[buf] + wh * TP + sub * PU + g;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float s = quad_sum(sum[n]);
            if (t == 0) out[8 * n] = s;
        }
        __syncthreads();
        for (int i = tid; i < TP && p0 + i < len; i += hw * nsub * 32) {
            float s = 0.f;
            for (int h = 0; h < hw; ++h) s += sums[buf][h * TP + i];
            if (i != tid && a.in && p0 + i < len - 1) old = a.in[score0 + i];
            a.out[score0 + i] = a.in && p0 + i < len - 1 ? fmaf(a.decay, old, s) : s;
        }
        r = r2;
        tile = tile2;
        len = len2;
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

// [head_dim 128][dtype]: the kernel, positions of a warp, CTAs of an SM
struct DecodeKernel {
    void (*run)(WeightArgs, int, int);
    int positions, ctas;
};
template <int D, int KV>
constexpr DecodeKernel decode_kernel() {
    return {weights_decode<D, KV>, Stream<D, KV>::PU, Stream<D, KV>::CTAS};
}
constexpr DecodeKernel decode_kernels[2][4] = {
    {decode_kernel<64, kKvF32>(), decode_kernel<64, 0>(), decode_kernel<64, 1>(), decode_kernel<64, 2>()},
    {decode_kernel<128, kKvF32>(), decode_kernel<128, 0>(), decode_kernel<128, 1>(), decode_kernel<128, 2>()}};

cudaError_t launch_decode(const DecodeKernel& k, const WeightArgs& a, int sms, cudaStream_t s) {
    // a warp per KV head up to eight, else several per head
    const int hw = std::min(a.Hkv, 8), nsub = 8 / hw, tp = k.positions * nsub;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms * k.ctas, a.B * (((int64_t)a.lim + tp - 1) / tp)));
    cfg.blockDim = dim3((unsigned)(hw * nsub * 32));
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k.run, a, hw, nsub);
}

// What a chunk call needs (host lengths that are not negative), or
// SGL_ERR_UNSUPPORTED: the same for the call and for the size of its workspace.
int chunk_plan(const sgl_attn_params* p, int window, TcPlan* plan) {
    if (p->dtype != SGL_DTYPE_F32) return tc_plan(p, window, plan);
    if (p->batch > 65535) return SGL_ERR_UNSUPPORTED;
    for (int32_t r = 0; r < p->batch; ++r)
        if ((int64_t)p->host_prefix_lens[r] + p->host_extend_lens[r] > kMaxLen) return SGL_ERR_UNSUPPORTED;
    return SGL_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

namespace sgl {
int check_params(const sgl_attn_params* p);
}

extern "C" {

int sgl_attn_weights_workspace_bytes(const sgl_attn_params* params, int32_t window, size_t* bytes) {
    const int st = sgl::check_params(params);
    if (st) return st;
    if (!bytes || window < 0) return SGL_ERR_INVALID_ARG;
    if (params->host_extend_lens && params->batch > 0) {
        if (!params->host_prefix_lens) return SGL_ERR_INVALID_ARG;
        for (int32_t r = 0; r < params->batch; ++r)
            if (params->host_prefix_lens[r] < 0 || params->host_extend_lens[r] < 0) return SGL_ERR_INVALID_ARG;
    }
    size_t n = sgl::kWsAlign;
    if (params->host_extend_lens) {
        TcPlan plan{};
        if (const int e = chunk_plan(params, window, &plan)) return e;
        n += (size_t)plan.items * 2048;
    }
    *bytes = n;
    return SGL_OK;
}

int sgl_attn_weights(const void* q, const float* lse, const void* k_pool, const int32_t* req_to_token, int64_t ld,
                     const int32_t* lens, const int32_t* extend_lens, const sgl_attn_params* params, int32_t window,
                     const float* scores_in, float* scores_out, int64_t scores_ld, float decay, void* workspace,
                     size_t ws_bytes, sgl_stream_t stream) {
    const int st = sgl::check_params(params);
    if (st) return st;
    const int32_t B = params->batch;
    if (ld < 0 || scores_ld < 0 || window < 0 || !(decay >= 0.f) || !std::isfinite(decay)) return SGL_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, sgl::kWsAlign) || ws_bytes < sgl::kWsAlign) return SGL_ERR_WORKSPACE;
    if (B == 0) return SGL_OK;
    if (!lens) return SGL_ERR_INVALID_ARG;
    const int64_t lim = std::min<int64_t>(std::min(ld, scores_ld), kMaxLen);
    int64_t rows = B, most = lim;
    TcPlan plan{};
    if (extend_lens) {
        if (!params->host_extend_lens || !params->host_prefix_lens) return SGL_ERR_INVALID_ARG;
        rows = most = 0;
        for (int32_t r = 0; r < B; ++r) {
            const int64_t p = params->host_prefix_lens[r], e = params->host_extend_lens[r];
            if (p < 0 || e < 0 || p + e > std::min(ld, scores_ld)) return SGL_ERR_INVALID_ARG;
            rows += e;
            most = std::max(most, p + e);
        }
        if (const int e = chunk_plan(params, window, &plan)) return e;
    }
    if (most == 0) return SGL_OK;
    if (!k_pool || !req_to_token || !scores_out || (rows > 0 && (!q || !lse))) return SGL_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_pool, 16)) return SGL_ERR_INVALID_ARG;
    const int d = params->head_dim, kind = params->dtype;
    WeightArgs a{};
    a.q = q;
    a.lse = lse;
    a.kp = static_cast<const uint8_t*>(k_pool);
    a.r2t = req_to_token;
    a.lens = lens;
    a.ext = extend_lens;
    a.in = decay > 0.f ? scores_in : nullptr;
    a.out = scores_out;
    a.ld = ld;
    a.scores_ld = scores_ld;
    a.num_slots = params->num_slots;
    a.n_rows = rows;
    a.err = static_cast<uint32_t*>(workspace);
    a.B = B;
    a.Hq = params->num_qo_heads;
    a.Hkv = params->num_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.window = window;
    a.lim = (int)lim;
    a.row_bytes = kind == SGL_DTYPE_BF16_FP4KV ? fp4_row_bytes(a.Hkv, d)
                                               : a.Hkv * d * (kind == SGL_DTYPE_F32 ? 4 : kind == SGL_DTYPE_BF16 ? 2 : 1);
    a.scale = params->sm_scale > 0.f ? params->sm_scale : 1.0f / std::sqrt(static_cast<float>(d));
    if (kind == SGL_DTYPE_BF16_FP8KV || kind == SGL_DTYPE_BF16_FP4KV) a.scale *= params->k_scale;
    a.decay = decay;
    auto s = reinterpret_cast<cudaStream_t>(stream);
    if (!extend_lens) {
        const auto* kernel = &decode_kernels[d == 128][kind];
        return cuda_status(launch_decode(*kernel, a, target_sms(params), s));
    }
    if (kind != SGL_DTYPE_F32) {
        if (ws_bytes < sgl::kWsAlign + (size_t)plan.items * 2048) return SGL_ERR_WORKSPACE;
        auto* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sgl::kWsAlign);
        const int kv = kind == SGL_DTYPE_BF16 ? 0 : kind == SGL_DTYPE_BF16_FP8KV ? 1 : 2;
        return cuda_status(static_cast<cudaError_t>(launch_weights_tc(a, kv, d, plan, partial, s)));
    }
    int C = 1;
    while (C < kF32Cluster && 2 * C <= a.Hkv) C *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)C;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((most + kF32Tile - 1) / kF32Tile), (unsigned)B, (unsigned)C);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = (size_t)(d == 64 ? f32_smem<64>() : f32_smem<128>());
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    static sgl::PerDevice ready;
    if (const int e = ready_here(ready, [] { return large_smem(weights_chunk_f32<128>, f32_smem<128>()); }))
        return cuda_status(static_cast<cudaError_t>(e));
    return cuda_status(cudaLaunchKernelEx(&cfg, d == 64 ? weights_chunk_f32<64> : weights_chunk_f32<128>, a));
}

}  // extern "C"
