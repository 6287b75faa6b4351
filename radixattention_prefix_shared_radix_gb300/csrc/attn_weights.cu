// The attention weights that cached tokens get from a call's queries, summed
// over query rows and heads, added to the scores that the tokens have gathered.
//
// With s = sm_scale <q, k_p> and the row's log-sum-exp L from the attention
// call, a weight is exp(s - L): no second softmax, one product Q K^T and one
// exponential per (row, head, position), and a sum over rows.  In base 2,
// 2^(s log2 e - hi) times the row's factor 2^(-lo), hi + lo = L log2 e: hi alone
// is off by up to half a unit of its last place (2^-20 at L near 10), and the
// factor costs nothing, since the sum over rows takes it as the multiplier of a
// fused multiply-add (0 for a row that saw nothing).

#include <algorithm>
#include <cmath>

#include "common.h"
#include "device_common.cuh"
#include "fp4.cuh"

namespace {

using namespace sgldev;

constexpr int kKvF32 = 3;                // pools by dtype, as elsewhere: 0 bf16, 1 E4M3, 2 4-bit rows

struct WeightArgs {
    const void* q;
    const float* lse;
    const uint8_t* kp;
    const int32_t* r2t;
    const int32_t *lens, *ext;           // ext null: decode
    const float* in;                     // null: zeros
    float* out;
    int64_t ld, scores_ld, num_slots, n_rows;
    uint32_t* err;
    int B, Hq, Hkv, G, window, lim, row_bytes;
    float scale, decay;                  // scale: of a product, to a power of 2
};

// What request r asks: rows [row, row + ask) of the queries, row i of which sees
// positions 0 .. p0 + i; its scores [0, total), those from `fresh` on beginning
// at 0.  ask 0: nothing to do (or lengths that the tables do not hold).
struct Asked {
    int total, ask, p0, fresh;
    int64_t row;
};
__device__ __forceinline__ Asked asked(const WeightArgs& a, int r, int64_t before, bool flag) {
    Asked x{0, 0, 0, 0, 0};
    const int len = __ldg(a.lens + r);
    if (!a.ext) {
        if (len < 0 || len > a.lim) {
            if (flag) atomicOr(a.err, 2u);
            return x;
        }
        return Asked{len, len > 0 ? 1 : 0, len - 1, len - 1, r};
    }
    const int e = __ldg(a.ext + r);
    if (len < 0 || e < 0 || (int64_t)len + e > a.lim || before + e > a.n_rows) {
        if (flag) atomicOr(a.err, 2u);
        return x;
    }
    const int ask = a.window > 0 ? min(a.window, e) : e;
    return Asked{len + e, ask, len + e - ask, len, before + e - ask};
}

// hi and 2^(-lo) of a row's log-sum-exp L: hi + lo = L log2 e, log2 e as the sum of two floats
__device__ __forceinline__ float2 lse_parts(float l) {
    constexpr float kLow = 1.92596299e-8f;
    if (l == -INFINITY) return make_float2(0.f, 0.f);
    const float hi = l * kLog2e;
    return make_float2(hi, ex2_ftz(-fmaf(l, kLow, fmaf(l, kLog2e, -hi))));
}

// ---------------------------------------------------------------------------
// Chunks, on CUDA cores: a CTA per (tile of 32 positions, request) takes every KV
// head and asking row, 32 rows at a time; a thread has one position and four
// rows of each 32.
// ---------------------------------------------------------------------------
template <int D, int KV>
__device__ __forceinline__ float4 key4(const WeightArgs& a, int64_t slot, int h, int c) {
    const uint8_t* row = a.kp + slot * a.row_bytes;
    float4 v;
    if constexpr (KV == kKvF32) {
        v = reinterpret_cast<const float4*>(row)[h * (D / 4) + c];
    } else if constexpr (KV == 0) {
        const uint2 w = reinterpret_cast<const uint2*>(row)[h * (D / 4) + c];
        v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xffff0000u));
    } else if constexpr (KV == 1) {
        uint32_t lo, hi;
        e4m3x4_to_f16(reinterpret_cast<const uint32_t*>(row)[h * (D / 4) + c], lo, hi);
        const float2 x = __half22float2(*reinterpret_cast<__half2*>(&lo)), y = __half22float2(*reinterpret_cast<__half2*>(&hi));
        v = make_float4(x.x, x.y, y.x, y.y);
    } else {
        const uint32_t w = *reinterpret_cast<const uint16_t*>(row + fp4_code_off(h, D) + 2 * c);
        uint32_t y[4];
        e2m1x8_to_f16(w, y);
        const float f = e4m3_value(row[fp4_scale_off(h, a.Hkv, D) + c / 4]);
        const float2 p = __half22float2(*reinterpret_cast<__half2*>(&y[0])), s = __half22float2(*reinterpret_cast<__half2*>(&y[1]));
        v = make_float4(p.x * f, p.y * f, s.x * f, s.y * f);
    }
    return v;
}

template <int D, int KV>
__global__ void __launch_bounds__(256) weights_plain(const __grid_constant__ WeightArgs a) {
    constexpr int RS = D + 4;            // (rows of 32 in distinct banks)
    __shared__ __align__(16) float sk[32 * RS], sq[32 * RS];
    __shared__ float2 sl[32];
    __shared__ int64_t before_s;
    const int r = blockIdx.y, tid = threadIdx.x, t0 = blockIdx.x * 32;
    if (tid < 32) {
        int64_t s = 0;
        if (a.ext)
            for (int b = tid; b < r; b += 32) s += max(__ldg(a.ext + b), 0);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) before_s = s;
    }
    __syncthreads();
    const Asked x = asked(a, r, before_s, tid == 0 && t0 == 0);
    if (t0 >= x.total) return;
    const int pos = t0 + (tid >> 3), sub = tid & 7;
    int64_t slot = -1;
    if (pos < x.total) {
        slot = __ldg(a.r2t + r * a.ld + pos);
        if (slot < 0 || slot >= a.num_slots) {
            if (sub == 0) atomicOr(a.err, 1u);
            slot = -1;
        }
    }
    float sum = 0.f;
    const int rows = x.ask * a.G;
    // (rows before the one that first sees the tile are passed over)
    const int row0 = max(t0 - x.p0, 0) * a.G & ~31;
    for (int h = 0; h < a.Hkv; ++h) {
        __syncthreads();
        for (int c = sub; c < D / 4; c += 8) {
            const float4 v = slot >= 0 ? key4<D, KV>(a, slot, h, c) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(&sk[(tid >> 3) * RS + 4 * c]) = v;
        }
        for (int b = row0; b < rows; b += 32) {
            __syncthreads();
            const int mine = b + (tid >> 3);
            const int64_t qrow = (x.row + mine / a.G) * a.Hq + h * a.G + mine % a.G;
            for (int c = sub; c < D / 4; c += 8) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine < rows) {
                    if constexpr (KV == kKvF32) {
                        v = reinterpret_cast<const float4*>(a.q)[qrow * (D / 4) + c];
                    } else {
                        const uint2 w = reinterpret_cast<const uint2*>(a.q)[qrow * (D / 4) + c];
                        v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                                        __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
                    }
                }
                *reinterpret_cast<float4*>(&sq[(tid >> 3) * RS + 4 * c]) = v;
            }
            if (sub == 0) sl[tid >> 3] = mine < rows ? lse_parts(a.lse[qrow]) : make_float2(0.f, 0.f);
            __syncthreads();
            float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 k = *reinterpret_cast<const float4*>(&sk[(tid >> 3) * RS + c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 y = *reinterpret_cast<const float4*>(&sq[(4 * i + (sub & 3) + 16 * (sub >> 2)) * RS + c]);
                    dot[i] = fmaf(k.x, y.x, fmaf(k.y, y.y, fmaf(k.z, y.z, fmaf(k.w, y.w, dot[i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * i + (sub & 3) + 16 * (sub >> 2);
                const float2 l = sl[row];
                // a row sees positions up to its own
                if (b + row < rows && pos <= x.p0 + (b + row) / a.G)
                    sum = fmaf(ex2_ftz(fmaf(dot[i], a.scale, -l.x)), l.y, sum);
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sub == 0 && pos < x.total) {
        if (slot < 0) sum = 0.f;
        const int64_t at = r * a.scores_ld + pos;
        a.out[at] = a.in && pos < x.fresh ? fmaf(a.decay, a.in[at], sum) : sum;
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
    *bytes = sgl::kWsAlign;
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
    const int64_t lim = std::min<int64_t>(std::min(ld, scores_ld), INT32_MAX / 2);
    int64_t rows = B, most = lim;
    if (extend_lens) {
        if (!params->host_extend_lens || !params->host_prefix_lens) return SGL_ERR_INVALID_ARG;
        rows = most = 0;
        for (int32_t r = 0; r < B; ++r) {
            const int64_t p = params->host_prefix_lens[r], e = params->host_extend_lens[r];
            if (p < 0 || e < 0 || p + e > std::min(ld, scores_ld)) return SGL_ERR_INVALID_ARG;
            if (p + e > lim) return SGL_ERR_UNSUPPORTED;
            rows += e;
            most = std::max(most, p + e);
        }
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
    a.scale = (params->sm_scale > 0.f ? params->sm_scale : 1.0f / std::sqrt(static_cast<float>(d))) * kLog2e;
    if (kind == SGL_DTYPE_BF16_FP8KV || kind == SGL_DTYPE_BF16_FP4KV) a.scale *= params->k_scale;
    a.decay = decay;
    auto s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((most + 31) / 32), (unsigned)B);
    if (B > 65535) return SGL_ERR_UNSUPPORTED;
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(a); };
    switch (kind) {
        case SGL_DTYPE_F32: d == 64 ? go(weights_plain<64, kKvF32>) : go(weights_plain<128, kKvF32>); break;
        case SGL_DTYPE_BF16: d == 64 ? go(weights_plain<64, 0>) : go(weights_plain<128, 0>); break;
        case SGL_DTYPE_BF16_FP8KV: d == 64 ? go(weights_plain<64, 1>) : go(weights_plain<128, 1>); break;
        default: d == 64 ? go(weights_plain<64, 2>) : go(weights_plain<128, 2>); break;
    }
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
