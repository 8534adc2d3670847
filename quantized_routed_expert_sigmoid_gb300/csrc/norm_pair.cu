// norm_pair.cu -- the norm behind a block, its gate and residual scale, and the norm before the
// next block, in one pass:
//   n = y / sqrt(mean y^2 + eps) * gamma_post     (or y)
//   r = res_scale * x + scale * gate * n
//   u = r / sqrt(mean r^2 + eps) * gamma_pre
// Bound: bytes.  x and y are read once and r and u written once; between the two means the row
// stays in the registers of the threads that share it (8 elements a thread and step, 16-byte
// accesses), so the second mean costs no second read.  Two forms:
// - norm_stream_kernel, rows of 4097 to 16384 elements that 16-byte accesses can read: a CTA per row
//   and as many CTAs as fit, each taking every (CTAs)-th row.  What bounds a row is latency (read, mean,
//   mean, write), so every thread copies its own elements of the next rows into shared memory (cp.async,
//   DEPTH rows ahead) while it computes; nothing but its own copies is waited for.
// - norm_pair_kernel, the others: narrow rows take one warp each (no barrier), others 128, 256
//   or 1024 threads.
// Measured: 4096 rows of 2048, fp32 stream, bf16 u: 22.3 us for 117 MB (17.6 us at the copy's rate); 512 rows
// of 7168, bf16, gated: 9.9 us (4.4 us); one row of 2048: 2.6 us, a launch and two means.
#include <algorithm>

#include "products.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float load1(const void* p, int type, int64_t i) {
    if (type == MOE_F32) return __ldg(reinterpret_cast<const float*>(p) + i);
    if (type == MOE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
// Eight elements from a 16-byte boundary.  ONCE: they are not read again.
template <bool ONCE = false>
__device__ __forceinline__ void load8(const void* p, int type, int64_t i, float (&v)[8]) {
    if (type == MOE_F32) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        const float4 a = ONCE ? __ldcs(q) : q[0], b = ONCE ? __ldcs(q + 1) : q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        return;
    }
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint4 w = ONCE ? __ldcs(q) : *q;
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
    wait_for_previous();
    allow_next();
    const int64_t t = (int64_t)blockIdx.x * (kThreads / TPR) + tid / TPR;
    const bool live = t < a.T;                           // (threads of the last CTA without a row join its barriers)
    if (TPR == 32 && !live) return;                      // (a warp a row: no barrier below)
    const int H = live ? a.H : 0;                        // elements that this thread's row has to read and write
    auto first = [&](int c) { return VEC ? (c * TPR + i0) * 8 : c * 8 * TPR + i0; };
    constexpr int kStep = VEC ? 1 : TPR;

    auto row_in = [&](const void* p, int type, int64_t stride, int c, float (&v)[8]) {
        if constexpr (VEC) {
            if (first(c) < H) load8<true>(p, type, t * stride + first(c), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first(c) + j * kStep < H) v[j] = load1(p, type, t * stride + first(c) + j * kStep);
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
    const float gt = live && a.gate && a.gate_col == 0 ? __ldg(a.gate + t * a.gate_row) : 1.0f;
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
                if (first(c) < H) load8(a.gate, MOE_F32, t * a.gate_row + first(c), f);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (first(c) + j * kStep < H) f[j] = __ldg(a.gate + t * a.gate_row + (first(c) + j * kStep) * a.gate_col);
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
                if (first(c) < H) store8(a.x_out, a.x_type, t * a.x_out_stride + first(c), r[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (first(c) + j * kStep < H)
                        store_value(a.x_out, a.x_type, t * a.x_out_stride + first(c) + j * kStep, r[c][j]);
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
            if (first(c) < H) store8(a.u, a.u_type, t * a.u_stride + first(c), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first(c) + j * kStep < H) store_value(a.u, a.u_type, t * a.u_stride + first(c) + j * kStep, f[j]);
        }
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Eight elements that this thread has copied to shared memory.
__device__ __forceinline__ void lds_row8(uint32_t a, int type, float (&v)[8]) {
    if (type == MOE_F32) {
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(a) : "memory");
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(a + 16) : "memory");
        return;
    }
    uint32_t u[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(a) : "memory");
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

// TPR threads a row, NC steps of 8 elements each; DEPTH rows copied ahead.  A ring slot holds, for each step, the
// threads' shares of x, then of y.
template <int TPR, int NC, int CTAS, int DEPTH>
__global__ void __launch_bounds__(TPR, CTAS) norm_stream_kernel(const __grid_constant__ NormPairArgs a) {
    constexpr int kWarps = TPR / 32;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float part[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bx = a.x_type == MOE_F32 ? 32 : 16, by = a.y_type == MOE_F32 ? 32 : 16;     // bytes of a share
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring), slot = (uint32_t)(NC * TPR * (bx + by));
    auto at_x = [&](int s, int c) { return base + s * slot + (c * TPR + tid) * bx; };
    auto at_y = [&](int s, int c) { return base + s * slot + NC * TPR * bx + (c * TPR + tid) * by; };
    auto first = [&](int c) { return (c * TPR + tid) * 8; };
    auto fetch = [&](int64_t t, int s) {                  // row t into slot s (always one group of copies)
        if (t < a.T) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (first(c) >= a.H) continue;
                const char* py = static_cast<const char*>(a.y) + (t * a.y_stride + first(c)) * (by >> 3);
                copy16(at_y(s, c), py);
                if (by == 32) copy16(at_y(s, c) + 16, py + 16);
                if (a.x) {
                    const char* px = static_cast<const char*>(a.x) + (t * a.x_stride + first(c)) * (bx >> 3);
                    copy16(at_x(s, c), px);
                    if (bx == 32) copy16(at_x(s, c) + 16, px + 16);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the sum over the row's threads; which: the two sums of a row use different places
    auto row_sum = [&](float v, int which) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) part[which][warp] = v;
        __syncthreads();
        v = lane < kWarps ? part[which][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    wait_for_previous();
    allow_next();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(blockIdx.x + (int64_t)d * gridDim.x, d);
    int s = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float gt = a.gate && a.gate_col == 0 ? __ldg(a.gate + t * a.gate_row) : 1.0f;
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        float r[NC][8], ss = 0.f, inv = 1.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = 0.f;
            if (first(c) < a.H) lds_row8(at_y(s, c), a.y_type, r[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
        }
        if (a.gamma_post) inv = 1.0f / sqrtf(row_sum(ss, 0) / (float)a.H + a.eps);
        ss = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (first(c) >= a.H) continue;
            float f[8];
            if (a.gamma_post) {
                load8(a.gamma_post, MOE_F32, first(c), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] = r[c][j] * inv * f[j];
            }
            if (a.gate && a.gate_col != 0) {
                load8(a.gate, MOE_F32, t * a.gate_row + first(c), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] *= f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = a.scale * (r[c][j] * gt);
            if (a.x) {
                lds_row8(at_x(s, c), a.x_type, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] = fmaf(a.res_scale, f[j], r[c][j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
            if (a.x_out) store8(a.x_out, a.x_type, t * a.x_out_stride + first(c), r[c]);
        }
        fetch(t + (int64_t)DEPTH * gridDim.x, s);         // (this thread has read its shares of the slot)
        if (++s == DEPTH) s = 0;
        if (a.u) {
            inv = 1.0f / sqrtf(row_sum(ss, 1) / (float)a.H + a.eps);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (first(c) >= a.H) continue;
                float f[8];
                load8(a.gamma_pre, MOE_F32, first(c), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = r[c][j] * inv * f[j];
                store8(a.u, a.u_type, t * a.u_stride + first(c), f);
            }
        }
        // part[] of a mean is written again after the next barrier of the other one; with a single
        // mean a row the writes of the next row have to wait
        if (!(a.gamma_post && a.u)) __syncthreads();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int TPR, int NC, int CTAS, int DEPTH>
cudaError_t launch_stream(const NormPairArgs& a, cudaStream_t s) {
    const int row = NC * TPR * ((a.x_type == MOE_F32 ? 32 : 16) + (a.y_type == MOE_F32 ? 32 : 16));
    constexpr int kMost = NC * TPR * 64 * DEPTH;          // two fp32 rows
    static_assert(kMost <= 227 * 1024 - 1024, "ring");
    static std::atomic<uint64_t> ready;
    int sms = 0;
    const void* fn = (const void*)norm_stream_kernel<TPR, NC, CTAS, DEPTH>;
    cudaError_t err = prepare_kernel(fn, kMost, ready, &sms);
    if (err != cudaSuccess) return err;
    const int per_sm = std::max(1, std::min(CTAS, 220 * 1024 / (row * DEPTH + 1024)));
    void* args[] = {const_cast<NormPairArgs*>(&a)};
    return launch_early(fn, dim3(std::min(a.T, sms * per_sm)), TPR, (size_t)row * DEPTH, s, args);
}

// VEC: the form with 16-byte accesses is there too (rows that launch_stream takes when they can be read so need it not).
template <int TPR, int NC, bool VEC = true>
cudaError_t launch(const NormPairArgs& a, bool vec, cudaStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kRows = kThreads / TPR;
    const unsigned grid = ((unsigned)a.T + kRows - 1) / kRows;           // (T up to 2^31 - 1)
    void* args[] = {const_cast<NormPairArgs*>(&a)};
    const void* fn = (const void*)norm_pair_kernel<TPR, NC, false>;
    if constexpr (VEC)
        if (vec) fn = (const void*)norm_pair_kernel<TPR, NC, true>;
    return launch_early(fn, dim3(grid), kThreads, 0, s, args);
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
    // (measured with 512 rows of 7168, bf16: 10.0 us streamed, 15.4 with 1024 threads a row and one row a
    // CTA; with 4096 fp32 rows of 2048: 29.9 us streamed, 22.3 without: short rows have CTAs enough in flight)
    if (vec && a.H > 4096 && a.H <= 8192) return launch_stream<512, 2, 2, 2>(a, s);
    if (vec && a.H > 8192 && a.H <= 16384) return launch_stream<1024, 2, 1, 1>(a, s);
    if (a.H <= 256) return launch<32, 1>(a, vec, s);
    if (a.H <= 512) return launch<32, 2>(a, vec, s);
    if (a.H <= 1024) return launch<128, 1>(a, vec, s);
    if (a.H <= 2048) return launch<256, 1>(a, vec, s);
    if (a.H <= 4096) return launch<256, 2>(a, vec, s);
    if (a.H <= 8192) return launch<1024, 1, false>(a, false, s);
    if (a.H <= 16384) return launch<1024, 2, false>(a, false, s);
    return launch<1024, 4>(a, vec, s);
}

}  // namespace moe
