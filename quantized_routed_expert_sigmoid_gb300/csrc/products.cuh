// products.cuh -- declarations shared by the products over dense and 4-bit experts and the norm pair: the
// calls' arguments as the kernels take them, and their launches.
#pragma once

#include "internal.cuh"

namespace moe {

// Norm behind a block, gate, residual and the norm before the next block (norm_pair.cu).
struct NormPairArgs {
    int T, H;
    const void* x;               // NULL: 0
    int x_type;                  // of x and x_out
    int64_t x_stride;
    const void* y;
    int y_type;
    int64_t y_stride;
    const float* gate;           // nullable; element (t, h) at t * gate_row + h * gate_col
    int64_t gate_row, gate_col;
    const float* gamma_post;     // nullable
    const float* gamma_pre;
    float eps, res_scale, scale;
    void* x_out;                 // nullable
    int64_t x_out_stride;
    void* u;                     // nullable
    int u_type;
    int64_t u_stride;
};
cudaError_t launch_norm_pair(const NormPairArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- grouped products, dense and 4-bit weights
// y[i] = W[e] v_i (or the gated pair with w1) for the sorted positions i of each expert e.
struct RowsArgs {
    const void* x;               // rows x_stride elements apart
    int64_t x_stride;
    const int32_t* sorted_pairs; // v_i = x[sorted_pairs[i] / k]; NULL: x[i]
    const int32_t* offsets;      // [E+1]; NULL: one expert over all P rows
    int E, k, P, N, K;           // K: sum length, N: outputs
    bool bf16;                   // type of x (and of dense weights): bf16, else fp16
    const void* w0;              // W (or its 4-bit codes)
    const void* w1;              // W_up, NULL: plain product
    int64_t row_stride, expert_stride;   // dense weights, elements
    bool in_out;                 // dense weights stored [K][N]
    int group;                   // 4-bit weights: group length, 0: dense
    const void* s0;              // scales [E][N][K/group], fp16 or bf16
    const void* s1;
    const uint8_t* z0;           // zero points, NULL: 8
    const uint8_t* z1;
    bool s_bf16;
    void* y;
    int y_type;
    int64_t y_stride;
    int32_t* status;             // nullable
};
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s);            // streams the weights (rows.cu)
cudaError_t launch_w4(const RowsArgs& a, cudaStream_t s);              // 4-bit weights (w4.cu)

// Element i of a tensor of a value type.
__device__ __forceinline__ void store_value(void* p, int type, int64_t i, float v) {
    if (type == MOE_F32) reinterpret_cast<float*>(p)[i] = v;
    else if (type == MOE_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}
// silu(g) u = g / (1 + e^-g) u, from e^-|g|, which does not overflow: g / (1 + e^-g) with an e^-g past the largest number is 0
// from g = -88.7 down, where silu is -2e-37 (and the quick division gives 0 from -87.3).  silu(g) is an fp32 number, below 2^-126
// with the spacing of the subnormal ones.  FAST, for 16-bit outputs: the quick exponential is off by at most
// 2 + 1.173 |g| units of 2^-23 (1.3e-5 at g = -88, a 39th of half a step of fp16), the quick division, by 1 to 2, by 2 units.
template <bool FAST>
__device__ __forceinline__ float silu_times(float g, float u) {
    const float z = FAST ? __expf(-fabsf(g)) : expf(-fabsf(g));
    const float top = g >= 0.f ? g : g * z;
    return (FAST ? __fdividef(top, 1.0f + z) : top / (1.0f + z)) * u;
}
constexpr int kMaxW4In = 32768;      // n_in of 4-bit weights: one staged row of x has to fit beside the ring
cudaError_t launch_grouped_dense(const RowsArgs& a, cudaStream_t s);   // tcgen05, dense weights (ggemm_dense.cu)

}  // namespace moe
