// norm_pair.cu -- the norm behind a block, its gate and residual scale, and the norm before the
// next block, in one pass:
//   n = y / sqrt(mean y^2 + eps) * gamma_post     (or y)
//   r = res_scale * x + scale * gate * n
//   u = r / sqrt(mean r^2 + eps) * gamma_pre
// Bound: bytes.  x and y are read once and r and u written once; between the two means the row
// stays in the registers of the threads that share it (8 elements a thread and step, 16-byte
// accesses), so the second mean costs no second read.  Narrow rows take one warp each (no
// barrier), wider ones 256 or 1024 threads.
#include "internal.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float load1(const void* p, int type, int64_t i) {
    if (type == MOE_F32) return __ldg(reinterpret_cast<const float*>(p) + i);
    if (type == MOE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, int type, int64_t i, float v) {
    if (type == MOE_F32) reinterpret_cast<float*>(p)[i] = v;
    else if (type == MOE_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}
// Eight elements from a 16-byte boundary.
__device__ __forceinline__ void load8(const void* p, int type, int64_t i, float (&v)[8]) {
    if (type == MOE_F32) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        return;
    }
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == MOE_BF16) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}
__device__ __forceinline__ void store8(void* p, int type, int64_t i, const float (&v)[8]) {
    if (type == MOE_F32) {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == MOE_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
}

// TPR threads share a row, NC steps of 8 elements each; VEC: 16-byte accesses (thread i of the row
// takes elements 8i .. of a step), else single elements, neighbouring threads neighbouring ones.
template <int TPR, int NC, bool VEC>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_pair_kernel(const __grid_constant__ NormPairArgs a) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kWarpsRow = TPR / 32;
    __shared__ float part[2][kThreads / 32];
    const int tid = threadIdx.x, i0 = tid % TPR, lane = tid & 31;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / TPR) + tid / TPR;
    if (TPR == 32 && t >= a.T) return;                   // (a warp a row: no barrier below)
    auto first = [&](int c) { return VEC ? (c * TPR + i0) * 8 : c * 8 * TPR + i0; };
    constexpr int kStep = VEC ? 1 : TPR;

    auto row_in = [&](const void* p, int type, int64_t stride, int c, float (&v)[8]) {
        if constexpr (VEC) {
            if (first(c) < a.H) load8(p, type, t * stride + first(c), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first(c) + j * kStep < a.H) v[j] = load1(p, type, t * stride + first(c) + j * kStep);
        }
    };
    auto vec_in = [&](const float* p, int c, float (&v)[8]) {     // a vector over the channels
        if constexpr (VEC) {
            if (first(c) < a.H) load8(p, MOE_F32, first(c), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first(c) + j * kStep < a.H) v[j] = __ldg(p + first(c) + j * kStep);
        }
    };
    // 1 / sqrt(mean + eps) of the row whose threads hold ss
    auto inv_rms = [&](float ss, int which) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (TPR > 32) {
            if (lane == 0) part[which][tid >> 5] = ss;
            __syncthreads();
            const int w0 = tid / TPR * kWarpsRow;
            float v = lane < kWarpsRow ? part[which][w0 + lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            ss = v;
        }
        return 1.0f / sqrtf(ss / (float)a.H + a.eps);
    };

    float r[NC][8], xv[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] = xv[c][j] = 0.f;
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) row_in(a.y, a.y_type, a.y_stride, c, r[c]);
    constexpr bool kEarly = NC * TPR < 4096;             // (beyond, x would not fit beside r in the registers)
    if (kEarly && a.x)
#pragma unroll
        for (int c = 0; c < NC; ++c) row_in(a.x, a.x_type, a.x_stride, c, xv[c]);
    float inv = 1.0f;
    if (a.gamma_post) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
        inv = inv_rms(ss, 0);
    }
    const float gt = a.gate && a.gate_col == 0 ? __ldg(a.gate + t * a.gate_row) : 1.0f;
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float f[8];
        if (a.gamma_post) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.f;
            vec_in(a.gamma_post, c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = r[c][j] * inv * f[j];
        }
        if (a.gate && a.gate_col != 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.f;
            if constexpr (VEC) {
                if (first(c) < a.H) load8(a.gate, MOE_F32, t * a.gate_row + first(c), f);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (first(c) + j * kStep < a.H) f[j] = __ldg(a.gate + t * a.gate_row + (first(c) + j * kStep) * a.gate_col);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] *= f[j];
        }
        if (!kEarly && a.x) row_in(a.x, a.x_type, a.x_stride, c, xv[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[c][j] = a.scale * (r[c][j] * gt);
            if (a.x) r[c][j] = fmaf(a.res_scale, xv[c][j], r[c][j]);
            // (elements past the row's end must not count: a NaN gate or inverse would reach them)
            if (first(c) + j * kStep < a.H) ss = fmaf(r[c][j], r[c][j], ss);
        }
    }
    if (a.x_out) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (VEC) {
                if (first(c) < a.H) store8(a.x_out, a.x_type, t * a.x_out_stride + first(c), r[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (first(c) + j * kStep < a.H)
                        store1(a.x_out, a.x_type, t * a.x_out_stride + first(c) + j * kStep, r[c][j]);
            }
        }
    }
    if (!a.u) return;
    inv = inv_rms(ss, 1);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float f[8] = {};
        vec_in(a.gamma_pre, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = r[c][j] * inv * f[j];
        if constexpr (VEC) {
            if (first(c) < a.H) store8(a.u, a.u_type, t * a.u_stride + first(c), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first(c) + j * kStep < a.H) store1(a.u, a.u_type, t * a.u_stride + first(c) + j * kStep, f[j]);
        }
    }
}

template <int TPR, int NC>
cudaError_t launch(const NormPairArgs& a, bool vec, cudaStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kRows = kThreads / TPR;
    const unsigned grid = (unsigned)((a.T + kRows - 1) / kRows);
    if (vec) norm_pair_kernel<TPR, NC, true><<<grid, kThreads, 0, s>>>(a);
    else norm_pair_kernel<TPR, NC, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

bool rows16(const void* p, int type, int64_t stride) {
    return !p || ((uintptr_t)p % 16 == 0 && stride * (type == MOE_F32 ? 4 : 2) % 16 == 0);
}

}  // namespace

cudaError_t launch_norm_pair(const NormPairArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    const bool vec = a.H % 8 == 0 && rows16(a.x, a.x_type, a.x_stride) && rows16(a.y, a.y_type, a.y_stride) &&
                     rows16(a.x_out, a.x_type, a.x_out_stride) && rows16(a.u, a.u_type, a.u_stride) &&
                     rows16(a.gamma_post, MOE_F32, 0) && rows16(a.gamma_pre, MOE_F32, 0) &&
                     (!a.gate || a.gate_col == 0 || (a.gate_col == 1 && rows16(a.gate, MOE_F32, a.gate_row)));
    if (a.H <= 256) return launch<32, 1>(a, vec, s);
    if (a.H <= 512) return launch<32, 2>(a, vec, s);
    if (a.H <= 2048) return launch<256, 1>(a, vec, s);
    if (a.H <= 4096) return launch<256, 2>(a, vec, s);
    if (a.H <= 8192) return launch<1024, 1>(a, vec, s);
    if (a.H <= 16384) return launch<1024, 2>(a, vec, s);
    return launch<1024, 4>(a, vec, s);
}

}  // namespace moe
