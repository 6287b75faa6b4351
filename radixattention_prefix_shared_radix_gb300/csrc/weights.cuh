// What the kernels that sum attention weights (attn_weights.cu, weights_tc.cu)
// share: their arguments, what a request asks, and a weight.
#pragma once

#include <algorithm>

#include "device_common.cuh"
#include "fp4.cuh"

namespace sgl {
namespace wts {

using namespace sgldev;

constexpr int kMaxLen = 1 << 26;         // positions of a context
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
    float scale, decay;                  // scale: of a product
};

// What request r asks of a chunk call: rows [row, row + ask) of the queries, row i
// of which sees positions 0 .. p0 + i; its scores [0, total), those from `fresh` on
// beginning at 0.  total 0: nothing to do (or lengths that the tables do not hold).
struct Asked {
    int total, ask, p0, fresh;
    int64_t row;
};
__device__ __forceinline__ Asked asked(const WeightArgs& a, int len, int ext, int64_t before) {
    if (len < 0 || ext < 0 || (int64_t)len + ext > a.lim || before + ext > a.n_rows) return Asked{0, 0, 0, 0, 0};
    const int ask = a.window > 0 ? min(a.window, ext) : ext;
    return Asked{len + ext, ask, len + ext - ask, len, before + ext - ask};
}

// What a row adds to its products' scale before the exponential: minus its
// log-sum-exp, and -infinity for a row that saw nothing (which is passed over
// besides: its products may be infinite or NaN).
__device__ __forceinline__ float minus_lse(float l) { return l == -INFINITY ? l : -l; }
// exp(s + m): the difference first, rounded once, then to base 2 (in base 2
// from the start the log-sum-exp itself would be rounded, by up to 2^-20)
__device__ __forceinline__ float weight_of(float product, float scale, float m) {
    return ex2_ftz(fmaf(product, scale, m) * kLog2e);
}

// Chunks on the tensor cores (weights_tc.cu): what a call needs of its
// workspace is 2048 bytes an item.
struct TcPlan {
    int64_t items, tiles;                // work items; tiles of 256 positions
    int run;                             // query blocks of an item
    int sms;                             // SMs to fill
};
// params->num_sms, or the device's SMs (bounded, so that products with it stay small)
inline int target_sms(const sgl_attn_params* p) { return std::min(query_num_sms(p->num_sms), 4096); }
int tc_plan(const sgl_attn_params* params, int window, TcPlan* plan);
// 0 or a cudaError_t
int launch_weights_tc(const WeightArgs& args, int kv, int head_dim, const TcPlan& plan, float* partial, cudaStream_t s);

}  // namespace wts
}  // namespace sgl
