// block_ops.cuh -- the operators around the routed experts (dense products with an epilogue, layer norm, balance
// loss): the calls' arguments as the kernels take them, their launches, and the rows' accesses that the norms share.
#pragma once

#include "products.cuh"

namespace moe {

// y = res_scale * r + scale * act(x W^T + bias) (linear.cu).
struct LinearArgs {
    int T, N, K;
    bool bf16;                   // type of x and W: bf16, else fp16
    const void* w;
    int64_t w_stride;
    bool in_out;                 // W stored [K][N]
    const void* bias;            // nullable
    int bias_type;
    int act;                     // MOE_ACT_*
    float scale, res_scale;
    const void* x;
    int64_t x_stride;
    const void* r;               // nullable
    int r_type;
    int64_t r_stride;
    void* y;
    int y_type;
    int64_t y_stride;
    int32_t* status;             // nullable
};
bool linear_pairs(const LinearArgs& a);                  // whether T rows take the kernel of CTA pairs
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);

// Layer norm and its gradient (layer_norm.cu).
struct LayerNormArgs {
    int T, H;
    const void* x;
    int x_type;                  // of x, add and dx
    int64_t x_stride;
    void* y;                     // forward: the output; backward: dy (read only)
    int y_type;
    int64_t y_stride;
    const float* gamma;          // nullable: 1
    const float* beta;           // nullable: 0
    float eps;
    float* mean;                 // [T] (forward: nullable)
    float* rstd;
    // backward
    const void* add;             // nullable
    int64_t add_stride;
    void* dx;
    int64_t dx_stride;
    float* dgamma;               // [H], nullable
    float* dbeta;
    bool accumulate;             // dgamma, dbeta += instead of =
    float* partial;              // [norm_partial_rows][2][H]
};
cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const LayerNormArgs& a, cudaStream_t s);
int norm_partial_rows(int T);    // rows of partial sums that the backward pass of T rows may write

// The router's balance loss (balance.cu).
struct BalanceArgs {
    int E, k, T, n_seqs;
    bool sigmoid, accumulate;
    float coef;
    const float* logits;
    int64_t stride;
    const int32_t* ids;
    const int32_t* seq_offsets;  // nullable
    const uint8_t* mask;         // nullable
    const float* upstream;       // nullable: 1
    float* loss;                 // nullable
    int32_t* counts;             // nullable
    float* dlogits;              // nullable
    int64_t dstride;
    int32_t* status;             // nullable
    void* ws;
};
size_t balance_ws_bytes(int E, int T, int n_seqs);
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s);

__device__ __forceinline__ float load1(const void* p, int type, int64_t i) {
    if (type == MOE_F32) return reinterpret_cast<const float*>(p)[i];
    if (type == MOE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
// Two 16-bit values of a word.
__device__ __forceinline__ float2 unpack2(uint32_t u, int type) {
    if (type == MOE_BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, int type) {
    if (type == MOE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// V neighbouring elements of a row (V = 1, or 4 or 8 of a pointer aligned to V elements, 16 bytes at most an access), which
// are not read again.
template <int V>
__device__ __forceinline__ void load_once(const void* p, int type, int64_t i, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = load1(p, type, i);
    } else if (type == MOE_F32) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const float4 a = __ldcs(q + j);
            v[4 * j] = a.x; v[4 * j + 1] = a.y; v[4 * j + 2] = a.z; v[4 * j + 3] = a.w;
        }
    } else {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
        uint32_t u[V / 2];
        if constexpr (V == 8) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4*>(q));
            u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
        } else {
            const uint2 w = __ldcs(reinterpret_cast<const uint2*>(q));
            u[0] = w.x; u[1] = w.y;
        }
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float2 f = unpack2(u[j], type);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}
// V neighbouring elements of an fp32 vector over the channels.
template <int V>
__device__ __forceinline__ void load_vec(const float* p, int i, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = __ldg(p + i);
    } else {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p + i) + j);
            v[4 * j] = a.x; v[4 * j + 1] = a.y; v[4 * j + 2] = a.z; v[4 * j + 3] = a.w;
        }
    }
}
template <int V>
__device__ __forceinline__ void store_row(void* p, int type, int64_t i, const float (&v)[V]) {
    if constexpr (V == 1) {
        store_value(p, type, i, v[0]);
    } else if (type == MOE_F32) {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
        uint16_t* q = reinterpret_cast<uint16_t*>(p) + i;
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(q) = make_uint4(pack2(v[0], v[1], type), pack2(v[2], v[3], type),
                                                      pack2(v[4], v[5], type), pack2(v[6], v[7], type));
        else *reinterpret_cast<uint2*>(q) = make_uint2(pack2(v[0], v[1], type), pack2(v[2], v[3], type));
    }
}

}  // namespace moe
