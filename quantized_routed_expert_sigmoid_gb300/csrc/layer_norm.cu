// layer_norm.cu -- layer norm, forward and backward:
//   m = mean x, r = 1 / sqrt(mean (x - m)^2 + eps), h = (x - m) r, y = h gamma + beta
//   g = dy gamma, dx = add + r (g - mean g - h mean(g h)), dgamma = sum_t dy h, dbeta = sum_t dy
// Bound: bytes.  A row is read once and stays in the registers of the threads that share it between its sums.
// A mean in fp32 is off by up to a few 2^-24 of the row's largest values, which is much of (x - m) where the
// row lies far from 0.  So the sum of (x - m) is taken along with that of its squares (no pass of its own) and the
// rest d = mean (x - m) is taken off: h = (x - m - d) r, the variance mean (x - m)^2 - d^2.  The backward pass, which gets
// the mean rounded to fp32, does the same.
// Kernels (times at 2048 channels, inputs from HBM):
// - forward_kernel, backward_kernel: a CTA an SM, 16 channels a thread, as many warps a row as it takes, the rows dealt to the
//   CTAs' groups of warps.  The types are the template's: with types looked up at every access the backward pass took 62
//   instructions an element, and those, not the bytes, were its bound (30.5 us for 4096 rows).  Arithmetic on
//   pairs of channels (fp32x2 instructions).  Rows whose addresses allow it (16 bytes of fp32 or 16-bit rows alone, 8 of 16-bit rows
//   among fp32 ones) come ahead through shared memory: every thread copies its own elements of the next rows (cp.async), and
//   nothing but its own copies is waited for.  Other rows are read element by element.
//   4096 rows, fp32 to bf16: forward 12.2 us, 4.1 TB/s (bytes alone: 7.4); backward with the residual's gradient 26.3 us,
//   4.5 TB/s (17.3).  512 rows of 7168, bf16: 15.7 us (3.3), 9.4 without the sums over the rows: two launches, four rows one after another.
//   1024 threads leave too few registers for rows, sums and gamma: slower.  Forward with gamma and beta in shared memory and two CTAs an
//   SM: 4096 rows of fp32 12.1 -> 11.8, of bf16 (bytes alone 4.9) 10.2 -> 12.7.
// - row_kernel: forward, a few rows (which leave most SMs without any): more threads a row, no ring to fill; and what the others
//   do not take: rows above 8192 elements, bf16 with fp16.  One row: 2.1 us, a launch and three trips to memory; 2048 rows of 12288,
//   fp32 to bf16: 50.8 us (22.3), 1024 of 16384, bf16: 33.6 (9.9).
// - wide_backward_kernel: the gradient of those, in the simplest form: element by element, types looked up, sums for gamma and beta
//   in memory.  2048 rows of 12288: 262 us (37), 1024 of 16384, bf16: 218 (15).
// - sums_kernel: dgamma and dbeta of the CTAs' partial sums.
#include <algorithm>

#include "block_ops.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- pairs of fp32 values
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum_of(F2 v) {
    const float2 f = split(v);
    return f.x + f.y;
}

// ---------------------------------------------------------------- elements of a type
template <typename T> __device__ __forceinline__ float value(T v);
template <> __device__ __forceinline__ float value<float>(float v) { return v; }
template <> __device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float value<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }
template <typename T> __device__ __forceinline__ F2 pair_of(uint32_t u) {
    const float2 f = unpack2(u, std::is_same<T, __nv_bfloat16>::value ? (int)MOE_BF16 : (int)MOE_F16);
    return pair(f.x, f.y);
}
template <typename T> __device__ __forceinline__ uint32_t packed(F2 v) {
    const float2 f = split(v);
    return pack2(f.x, f.y, std::is_same<T, __nv_bfloat16>::value ? (int)MOE_BF16 : (int)MOE_F16);
}
// V neighbouring elements (V >= 4) as pairs, from shared memory and to a row.
template <typename T, int V>
__device__ __forceinline__ void from_shared(uint32_t at, F2 (&v)[V / 2]) {
    if constexpr (sizeof(T) == 4) {
        asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(at) : "memory");
    } else if constexpr (V == 4) {
        uint32_t u[2];
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "r"(at) : "memory");
        v[0] = pair_of<T>(u[0]);
        v[1] = pair_of<T>(u[1]);
    } else {
        uint32_t u[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at) : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pair_of<T>(u[j]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void to_row(T* p, const F2 (&v)[V / 2]) {
    if constexpr (sizeof(T) == 4) {
        asm volatile("st.global.v2.b64 [%0], {%1,%2};" ::"l"(p), "l"(v[0]), "l"(v[1]) : "memory");
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(packed<T>(v[0]), packed<T>(v[1]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(packed<T>(v[0]), packed<T>(v[1]), packed<T>(v[2]), packed<T>(v[3]));
    }
}
template <int BYTES>
__device__ __forceinline__ void copy_ahead(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// ---------------------------------------------------------------- rows shared by warps
constexpr int kThreads = 512, kWarps = kThreads / 32, kChannels = 16, kPairs = kChannels / 2;

// Sums of four values over the `warps` warps of a row, all of whose threads get the same bits.  part: [warps] of the row, not
// in use by sums that some of them may still read; barrier: the row's own.  Within a warp lanes trade what they do not keep: after
// two steps a lane holds one of the four.
__device__ __forceinline__ float4 row_sums(float a0, float a1, float a2, float a3, float4* part, int w, int warps, int barrier) {
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16, odd = lane & 8;
    float k0 = hi ? a2 : a0, k1 = hi ? a3 : a1;
    k0 += __shfl_xor_sync(0xffffffffu, hi ? a0 : a2, 16);
    k1 += __shfl_xor_sync(0xffffffffu, hi ? a1 : a3, 16);
    float v = odd ? k1 : k0;
    v += __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    if ((lane & 7) == 0) reinterpret_cast<float*>(part + w)[lane >> 3] = v;
    if (warps > 1) asm volatile("barrier.cta.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
    else __syncwarp();
    float4 s = part[0];
#pragma unroll 4
    for (int i = 1; i < warps; ++i) {
        const float4 f = part[i];
        s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
    }
    return s;
}
__device__ __forceinline__ float row_sum(float a, float* part, int w, int warps, int barrier) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (warps == 1) return a;
    if ((threadIdx.x & 31) == 0) part[w] = a;
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
    a = part[0];
#pragma unroll 4
    for (int i = 1; i < warps; ++i) a += part[i];
    return a;
}

struct NormParams {
    LayerNormArgs a;
    int warps;                   // of a row
    int depth;                   // rows copied ahead: 2 or 4
};
// Where a thread stands: its row group, its place in it, the channels that it has (V at a time, V * 32 * warps apart).
struct Place {
    int group, w, first, step;
    bool idle;
    __device__ __forceinline__ Place(int warps, int V) {
        const int warp = threadIdx.x >> 5;
        group = warp / warps;
        w = warp - group * warps;
        first = (w * 32 + (threadIdx.x & 31)) * V;
        step = 32 * warps * V;
        idle = group >= kWarps / warps;
    }
};
__device__ __forceinline__ void wait_ahead(int depth) {
    if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
template <typename T>
__device__ __forceinline__ void load_pairs(const T* row, const Place& at, int H, F2 (&v)[kPairs], float none) {
    // (element by element: V = 1)
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        const int e0 = at.first + 2 * j * at.step, e1 = e0 + at.step;
        v[j] = pair(e0 < H ? value<T>(row[e0]) : none, e1 < H ? value<T>(row[e1]) : none);
    }
}
// gamma or beta of a thread's channels (`none` without one).
template <int V>
__device__ __forceinline__ void load_channels(const float* p, const Place& at, int H, float none, F2 (&v)[kPairs]) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = pair(none, none);
    if (!p) return;
    if constexpr (V == 1) {
        load_pairs<float>(p, at, H, v, 0.f);
    } else {
#pragma unroll
        for (int c = 0; c < kChannels / V; ++c)
            if (at.first + c * at.step < H) {
                float f[V];
                load_vec<V>(p, at.first + c * at.step, f);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) v[c * (V / 2) + j] = pair(f[2 * j], f[2 * j + 1]);
            }
    }
}

// ---------------------------------------------------------------- forward
// FULL: the row's threads have all their channels (H = 512 warps): nothing is compared with the row's end.
template <typename X, typename Y, int V, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) forward_kernel(const __grid_constant__ NormParams p) {
    constexpr int NC = kChannels / V, kBytes = V * sizeof(X), kSlot = kThreads * NC * kBytes;
    const LayerNormArgs& a = p.a;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float one[2][kWarps];
    __shared__ float4 four[2][kWarps];
    const Place at(p.warps, V);
    const int tid = threadIdx.x, groups = kWarps / p.warps, g0 = at.group * p.warps;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + tid * kBytes;
    const int every = gridDim.x * groups, T = a.T;
    auto here = [&](int c) { return FULL || at.first + c * at.step < a.H; };
    wait_for_previous();
    allow_next();
    if (at.idle) return;
    int t = blockIdx.x + gridDim.x * at.group, ahead = t;
    const X* x_next = static_cast<const X*>(a.x) + (int64_t)t * a.x_stride + (V > 1 ? at.first : 0);
    Y* y_out = static_cast<Y*>(a.y) + (int64_t)t * a.y_stride + (V > 1 ? at.first : 0);
    const int64_t x_step = every * a.x_stride, y_step = every * a.y_stride;
    auto fetch = [&](int s) {                             // the next row into slot s (always one group of copies)
        if constexpr (V > 1) {
            if (ahead < T) {
                const X* src = x_next;
#pragma unroll
                for (int c = 0; c < NC; ++c, src += at.step)
                    if (here(c)) copy_ahead<kBytes>(mine + s * kSlot + c * kThreads * kBytes, src);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ahead += every;                               // (T + 5 * every < 2^31)
            x_next += x_step;
        }
    };
    for (int d = 0; V > 1 && d < p.depth; ++d) fetch(d);
    F2 gamma[kPairs], beta[kPairs];
    load_channels<V>(a.gamma, at, a.H, 1.f, gamma);
    load_channels<V>(a.beta, at, a.H, 0.f, beta);
    const float inv = 1.0f / (float)a.H;
    int turn = 0, s = 0;
    for (; t < T; t += every, turn ^= 1, y_out += y_step) {
        F2 x[kPairs];
        if constexpr (V > 1) {
            wait_ahead(p.depth);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                F2 v[V / 2];
                if (!FULL)
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) v[j] = 0;
                if (here(c)) from_shared<X, V>(mine + s * kSlot + c * kThreads * kBytes, v);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) x[c * (V / 2) + j] = v[j];
            }
            fetch(s);                                     // (this thread has read its share of the slot)
            if (++s == p.depth) s = 0;
        } else {
            load_pairs<X>(x_next, at, a.H, x, 0.f);
            x_next += x_step;
        }
        F2 sum = x[0];
#pragma unroll
        for (int i = 1; i < kPairs; ++i) sum = add2(sum, x[i]);
        const float m = row_sum(sum_of(sum), one[turn] + g0, at.w, p.warps, 1 + at.group) * inv;
        const F2 minus = pair(-m, -m);
        F2 q0 = 0, q1 = 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            x[i] = add2(x[i], minus);
            // (what lies behind the row's end is 0, which must not count)
            if constexpr (V > 1) {
                if (!here(i / (V / 2))) x[i] = 0;
            } else {
                const int e0 = at.first + 2 * i * at.step;
                if (e0 + at.step >= a.H) x[i] = e0 < a.H ? pair(split(x[i]).x, 0.f) : 0;
            }
            q0 = add2(q0, x[i]);
            q1 = fma2(x[i], x[i], q1);
        }
        const float4 q = row_sums(sum_of(q0), sum_of(q1), 0.f, 0.f, four[turn] + g0, at.w, p.warps, 1 + at.group);
        const float d = q.x * inv;
        float var = q.y * inv - d * d;
        if (var < 0.f) var = 0.f;                         // (a NaN stays)
        const float r = rsqrtf(var + a.eps);
        if (at.w == 0 && (tid & 31) == 0) {
            if (a.mean) a.mean[t] = m + d;
            if (a.rstd) a.rstd[t] = r;
        }
        if (!a.y) continue;
        const F2 scale = pair(r, r), shift = pair(-d, -d);
        if constexpr (V > 1) {
            Y* out = y_out;
#pragma unroll
            for (int c = 0; c < NC; ++c, out += at.step) {
                if (!here(c)) continue;
                F2 v[V / 2];
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const int i = c * (V / 2) + j;
                    v[j] = fma2(mul2(add2(x[i], shift), scale), gamma[i], beta[i]);
                }
                to_row<Y, V>(out, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float2 v = split(fma2(mul2(add2(x[i], shift), scale), gamma[i], beta[i]));
                const int e0 = at.first + 2 * i * at.step;
                if (e0 < a.H) y_out[e0] = rounded<Y>(v.x);
                if (e0 + at.step < a.H) y_out[e0 + at.step] = rounded<Y>(v.y);
            }
        }
    }
    if constexpr (V > 1) asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- backward
// A thread keeps the sums for gamma and beta of its channels in registers; the CTA's groups join theirs in shared memory and
// write one row of partial sums, which sums_kernel adds in a fixed order.
template <typename X, typename Y, int V, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) backward_kernel(const __grid_constant__ NormParams p) {
    constexpr int NC = kChannels / V, kX = V * sizeof(X), kY = V * sizeof(Y);
    constexpr int kOffY = kThreads * NC * kX, kOffAdd = kOffY + kThreads * NC * kY;
    const LayerNormArgs& a = p.a;
    extern __shared__ __align__(16) float shared[];       // the ring, then the groups' sums
    __shared__ float4 four[2][kWarps];
    const Place at(p.warps, V);
    const int tid = threadIdx.x, groups = kWarps / p.warps, g0 = at.group * p.warps;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(shared), slot = kOffAdd + (a.add ? kOffY : 0);
    const int every = gridDim.x * groups, T = a.T;
    auto here = [&](int c) { return FULL || at.first + c * at.step < a.H; };
    wait_for_previous();
    allow_next();
    int t = at.idle ? T : blockIdx.x + gridDim.x * at.group, ahead = t;
    const int off = V > 1 ? at.first : 0;
    // (rows by their number each time: pointers and strides kept for four of them would not fit the registers)
    auto x_row = [&](int t) { return static_cast<const X*>(a.x) + (t * a.x_stride + off); };
    auto dy_row = [&](int t) { return static_cast<const Y*>(a.y) + (t * a.y_stride + off); };
    auto add_row = [&](int t) { return static_cast<const X*>(a.add) + (t * a.add_stride + off); };
    auto fetch = [&](int s) {                             // the next row into slot s (always one group of copies)
        if constexpr (V > 1) {
            if (ahead < T) {
                const uint32_t dst = ring + s * slot;
                const X* px = x_row(ahead);
                const Y* py = dy_row(ahead);
#pragma unroll
                for (int c = 0; c < NC; ++c, px += at.step, py += at.step) {
                    if (!here(c)) continue;
                    copy_ahead<kX>(dst + (c * kThreads + tid) * kX, px);
                    copy_ahead<kY>(dst + kOffY + (c * kThreads + tid) * kY, py);
                }
                if (a.add) {
                    const X* pa = add_row(ahead);
#pragma unroll
                    for (int c = 0; c < NC; ++c, pa += at.step)
                        if (here(c)) copy_ahead<kX>(dst + kOffAdd + (c * kThreads + tid) * kX, pa);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ahead += every;                               // (T + 5 * every < 2^31)
        }
    };
    for (int d = 0; V > 1 && d < p.depth; ++d) fetch(d);
    float m = t < T ? __ldg(a.mean + t) : 0.f, r = t < T ? __ldg(a.rstd + t) : 0.f;
    F2 gamma[kPairs], sg[kPairs], sb[kPairs];
    load_channels<V>(a.gamma, at, a.H, 1.f, gamma);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) sg[i] = sb[i] = 0;
    const float inv = 1.0f / (float)a.H;
    int turn = 0, s = 0;
    for (; t < T; t += every, turn ^= 1) {
        F2 x[kPairs], dy[kPairs];
        if constexpr (V > 1) {
            wait_ahead(p.depth);
            const uint32_t src = ring + s * slot;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                F2 u[V / 2], v[V / 2];
                if (!FULL)
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) { u[j] = pair(m, m); v[j] = 0; }
                if (here(c)) {
                    from_shared<X, V>(src + (c * kThreads + tid) * kX, u);
                    from_shared<Y, V>(src + kOffY + (c * kThreads + tid) * kY, v);
                }
#pragma unroll
                for (int j = 0; j < V / 2; ++j) { x[c * (V / 2) + j] = u[j]; dy[c * (V / 2) + j] = v[j]; }
            }
        } else {
            load_pairs<X>(x_row(t), at, a.H, x, m);
            load_pairs<Y>(dy_row(t), at, a.H, dy, 0.f);
        }
        // (the next row's, early: their latency passes behind this one's sums)
        const bool more = t + every < T;
        const float next_m = more ? __ldg(a.mean + t + every) : 0.f, next_r = more ? __ldg(a.rstd + t + every) : 0.f;
        const F2 minus = pair(-m, -m);
        F2 q0 = 0, q1 = 0, q2 = 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {                // (x - m = dy = 0 behind the row's end)
            x[i] = add2(x[i], minus);
            const F2 g = mul2(dy[i], gamma[i]);
            q0 = add2(q0, g);
            q1 = fma2(g, x[i], q1);
            q2 = add2(q2, x[i]);
        }
        const float4 q = row_sums(sum_of(q0), sum_of(q1), sum_of(q2), 0.f, four[turn] + g0, at.w, p.warps, 1 + at.group);
        // h = x r - d r, dx = g r - m1 r - h m2 r (+ add)
        const float d = q.z * inv, c1 = -q.x * inv * r, c2 = -(q.y - d * q.x) * r * inv * r;
        const F2 rr = pair(r, r), dd = pair(-d, -d), m1 = pair(c1, c1), m2 = pair(c2, c2);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {                // (from here on x holds dx)
            const F2 h = mul2(add2(x[i], dd), rr);
            sg[i] = fma2(dy[i], h, sg[i]);
            sb[i] = add2(sb[i], dy[i]);
            x[i] = fma2(mul2(dy[i], gamma[i]), rr, fma2(h, m2, m1));
        }
        if (a.dx) {
            X* out = static_cast<X*>(a.dx) + (t * a.dx_stride + off);
            if constexpr (V > 1) {
                if (a.add) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (here(c)) {
                            F2 v[V / 2];
                            from_shared<X, V>(ring + s * slot + kOffAdd + (c * kThreads + tid) * kX, v);
#pragma unroll
                            for (int j = 0; j < V / 2; ++j) x[c * (V / 2) + j] = add2(v[j], x[c * (V / 2) + j]);
                        }
                }
#pragma unroll
                for (int c = 0; c < NC; ++c, out += at.step) {
                    if (!here(c)) continue;
                    F2 v[V / 2];
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) v[j] = x[c * (V / 2) + j];
                    to_row<X, V>(out, v);
                }
            } else {
                if (a.add) {
                    F2 v[kPairs];
                    load_pairs<X>(add_row(t), at, a.H, v, 0.f);
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) x[i] = add2(x[i], v[i]);
                }
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const float2 v = split(x[i]);
                    const int e0 = at.first + 2 * i * at.step;
                    if (e0 < a.H) out[e0] = rounded<X>(v.x);
                    if (e0 + at.step < a.H) out[e0 + at.step] = rounded<X>(v.y);
                }
            }
        }
        fetch(s);                                         // (this thread has read its shares of the slot)
        if (++s == p.depth) s = 0;
        m = next_m;
        r = next_r;
    }
    if constexpr (V > 1) asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.partial) return;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.H;
    // this thread's sums to the vectors of gamma's and beta's
    auto put = [&](float* g, float* b, int end) {
        if constexpr (V > 1) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const int e = at.first + (2 * i / V) * at.step + 2 * i % V;
                if (e >= end) continue;
                *reinterpret_cast<ulonglong2*>(g + e) = make_ulonglong2(sg[i], sg[i + 1]);
                *reinterpret_cast<ulonglong2*>(b + e) = make_ulonglong2(sb[i], sb[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float2 u = split(sg[i]), v = split(sb[i]);
                const int e0 = at.first + 2 * i * at.step, e1 = e0 + at.step;
                if (e0 < end) { g[e0] = u.x; b[e0] = v.x; }
                if (e1 < end) { g[e1] = u.y; b[e1] = v.y; }
            }
        }
    };
    if (groups == 1) {
        if (!at.idle) put(out, out + a.H, a.H);
        return;
    }
    __syncthreads();                                      // (everyone has read its last rows)
    const int width = kChannels * 32 * p.warps;           // [gamma, beta][group][width]
    if (!at.idle) put(shared + at.group * width, shared + (groups + at.group) * width, width);
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < 2 * a.H; i += kThreads) {
        const int which = i >= a.H;
        const float* from = shared + which * groups * width + (i - which * a.H);
        float v = 0.f;
        for (int g = 0; g < groups; ++g) v += from[g * width];
        out[i] = v;
    }
}

// ---------------------------------------------------------------- forward, a few rows, or rows of any kind
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
// Sums of v over the CTA.  part: [N][32], not in use by sums that some warps may still read.
template <int TPR, int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float* part) {
    warp_sums(v);
    const int lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i * 32 + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < TPR / 32 ? part[i * 32 + lane] : 0.f;
    warp_sums(v);
}

// A CTA of TPR threads a row, NC steps of V elements each.
template <int V, int TPR, int NC>
__global__ void __launch_bounds__(TPR) row_kernel(const __grid_constant__ LayerNormArgs a) {
    __shared__ float part[2][2 * 32];
    wait_for_previous();
    allow_next();
    const int64_t t = blockIdx.x;
    auto first = [&](int c) { return (c * TPR + (int)threadIdx.x) * V; };
    float x[NC][V], s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[c][j] = 0.f;
        if (first(c) < a.H) load_once<V>(a.x, a.x_type, t * a.x_stride + first(c), x[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] += x[c][j];
    cta_sums<TPR>(s, part[0]);
    const float m = s[0] / (float)a.H;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (first(c) < a.H)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[c][j] -= m;
                q[0] += x[c][j];
                q[1] = fmaf(x[c][j], x[c][j], q[1]);
            }
    cta_sums<TPR>(q, part[1]);
    const float d = q[0] / (float)a.H;
    float var = q[1] / (float)a.H - d * d;
    if (var < 0.f) var = 0.f;                            // (a NaN stays)
    const float r = rsqrtf(var + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[t] = m + d;
        if (a.rstd) a.rstd[t] = r;
    }
    if (!a.y) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (first(c) >= a.H) continue;
        float f[V], b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) { f[j] = 1.f; b[j] = 0.f; }
        if (a.gamma) load_vec<V>(a.gamma, first(c), f);
        if (a.beta) load_vec<V>(a.beta, first(c), b);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = fmaf((x[c][j] - d) * r, f[j], b[j]);
        store_row<V>(a.y, a.y_type, t * a.y_stride + first(c), f);
    }
}
template <int V, int TPR, int NC>
cudaError_t launch_row(const LayerNormArgs& a, cudaStream_t s) {
    void* args[] = {const_cast<LayerNormArgs*>(&a)};
    return launch_early((const void*)row_kernel<V, TPR, NC>, dim3((unsigned)a.T), TPR, 0, s, args);
}
template <int V>
cudaError_t rows_of(const LayerNormArgs& a, cudaStream_t s) {
    if (a.H <= 1024) return launch_row<V, 128, 8 / V>(a, s);
    if (a.H <= 2048) return launch_row<V, 256, 8 / V>(a, s);
    if (a.H <= 8192) return launch_row<V, 1024, 8 / V>(a, s);
    return launch_row<V, 1024, 32 / V>(a, s);
}

// ---------------------------------------------------------------- backward, rows of any kind
// A row is read twice (the second time from L1 and L2) and its share of the sums for gamma and beta added to the CTA's row of
// partial sums in memory.
__global__ void __launch_bounds__(1024) wide_backward_kernel(const __grid_constant__ LayerNormArgs a) {
    __shared__ float part[2][3 * 32];
    const int tid = threadIdx.x;
    wait_for_previous();
    allow_next();
    const float inv = 1.0f / (float)a.H;
    float* out = a.partial ? a.partial + (int64_t)blockIdx.x * 2 * a.H : nullptr;
    int turn = 0;
    bool begun = false;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const float m = __ldg(a.mean + t), r = __ldg(a.rstd + t);
        float q[3] = {0.f, 0.f, 0.f};
#pragma unroll 4
        for (int i = tid; i < a.H; i += 1024) {
            const float x = load1(a.x, a.x_type, t * a.x_stride + i) - m;
            const float g = load1(a.y, a.y_type, t * a.y_stride + i) * (a.gamma ? __ldg(a.gamma + i) : 1.f);
            q[0] += g;
            q[1] = fmaf(g, x, q[1]);
            q[2] += x;
        }
        cta_sums<1024>(q, part[turn]);
        const float d = q[2] * inv, m1 = q[0] * inv, m2 = (q[1] - d * q[0]) * r * inv;
#pragma unroll 4
        for (int i = tid; i < a.H; i += 1024) {
            const float h = (load1(a.x, a.x_type, t * a.x_stride + i) - m - d) * r, dy = load1(a.y, a.y_type, t * a.y_stride + i);
            if (out) {
                out[i] = begun ? fmaf(dy, h, out[i]) : dy * h;
                out[a.H + i] = begun ? out[a.H + i] + dy : dy;
            }
            if (a.dx) {
                float o = r * (dy * (a.gamma ? __ldg(a.gamma + i) : 1.f) - m1 - h * m2);
                if (a.add) o += load1(a.add, a.x_type, t * a.add_stride + i);
                store_value(a.dx, a.x_type, t * a.dx_stride + i, o);
            }
        }
        begun = true;
    }
}

// dgamma, dbeta: the sums of the partial rows, 32 V channels a CTA (blockIdx.y: gamma or beta), its W warps take turns at the rows.
// (One channel a lane and 32 warps while that is few CTAs: 1 us less at H = 2048, 0.5 more at 7168.)
template <int V, int W>
__global__ void __launch_bounds__(32 * W) sums_kernel(const float* partial, int rows, int H, float* dgamma, float* dbeta,
                                                               bool accumulate) {
    __shared__ float part[W][32 * V];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h0 = blockIdx.x * 32 * V;
    float* out = blockIdx.y ? dbeta : dgamma;
    wait_for_previous();
    allow_next();
    if (!out) return;
    float v[V] = {};
    if (h0 + lane * V < H) {
        const float* from = partial + (int64_t)blockIdx.y * H + h0 + lane * V;
#pragma unroll 10
        for (int i = w; i < rows; i += W) {
            float f[V];
            load_once<V>(from + (int64_t)2 * i * H, MOE_F32, 0, f);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] += f[j];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) part[w][lane * V + j] = v[j];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < 32 * V && h0 + c < H) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) s += part[i][c];
        out[h0 + c] = accumulate ? out[h0 + c] + s : s;
    }
}

constexpr int kMostPartials = 512, kMostHere = 32 * kWarps * kChannels;     // channels of a row of the kernels above
constexpr int kMostShared = 2 * kThreads * kChannels * 12;                  // two rows a group of fp32 x, dy and add: 192 KB

// V elements of these rows can be read at once.
bool aligned_rows(const void* p, int type, int64_t stride, int v) {
    const int64_t bytes = (type == MOE_F32 ? 4 : 2) * v, whole = bytes > 16 ? 16 : bytes;
    return !p || ((uintptr_t)p % whole == 0 && stride * (type == MOE_F32 ? 4 : 2) % whole == 0);
}
bool all_aligned(const LayerNormArgs& a, int v) {
    return a.H % v == 0 && aligned_rows(a.x, a.x_type, a.x_stride, v) && aligned_rows(a.y, a.y_type, a.y_stride, v) &&
           aligned_rows(a.add, a.x_type, a.add_stride, v) && aligned_rows(a.dx, a.x_type, a.dx_stride, v) &&
           aligned_rows(a.gamma, MOE_F32, 0, v) && aligned_rows(a.beta, MOE_F32, 0, v);
}

template <typename X, typename Y, int V>
cudaError_t launch_typed(const LayerNormArgs& a, bool backward, int grid, cudaStream_t s) {
    static std::atomic<uint64_t> ready[4];
    const bool full = V > 1 && a.H % (32 * kChannels) == 0;
    int sms = 0;
    const void* fn = backward ? (full ? (const void*)backward_kernel<X, Y, V, V != 1> : (const void*)backward_kernel<X, Y, V, false>)
                              : (full ? (const void*)forward_kernel<X, Y, V, V != 1> : (const void*)forward_kernel<X, Y, V, false>);
    cudaError_t err = prepare_kernel(fn, kMostShared, ready[2 * full + backward], &sms);
    if (err != cudaSuccess) return err;
    NormParams p{a, (a.H + 32 * kChannels - 1) / (32 * kChannels), 2};
    const int slot = kThreads * kChannels * (int)(backward ? sizeof(X) + sizeof(Y) + (a.add ? sizeof(X) : 0) : sizeof(X));
    if (4 * slot <= kMostShared) p.depth = 4;
    const int join = backward ? 2 * kThreads * kChannels * 4 : 0;
    void* args[] = {&p};
    return launch_early(fn, dim3(std::min(a.T, grid)), kThreads, std::max(V > 1 ? p.depth * slot : 0, join), s, args);
}
// The kernels for rows of these types; *none: there is none for them.
template <typename X, typename Y>
cudaError_t launch_pair_of(const LayerNormArgs& a, bool backward, int grid, cudaStream_t s) {
    if constexpr (sizeof(X) == 2 && sizeof(Y) == 2)
        if (all_aligned(a, 8)) return launch_typed<X, Y, 8>(a, backward, grid, s);
    if (all_aligned(a, 4)) return launch_typed<X, Y, 4>(a, backward, grid, s);
    return launch_typed<X, Y, 1>(a, backward, grid, s);
}
cudaError_t launch_rows(const LayerNormArgs& a, bool backward, int grid, cudaStream_t s, bool* none) {
    using B = __nv_bfloat16;
    const int x = a.x_type, y = a.y_type;
    *none = a.H > kMostHere;
    if (*none) return cudaSuccess;
    if (x == MOE_F32) {
        if (y == MOE_F32) return launch_pair_of<float, float>(a, backward, grid, s);
        return y == MOE_BF16 ? launch_pair_of<float, B>(a, backward, grid, s) : launch_pair_of<float, __half>(a, backward, grid, s);
    }
    if (x == MOE_BF16 && y != MOE_F16)
        return y == MOE_BF16 ? launch_pair_of<B, B>(a, backward, grid, s) : launch_pair_of<B, float>(a, backward, grid, s);
    if (x == MOE_F16 && y != MOE_BF16)
        return y == MOE_F16 ? launch_pair_of<__half, __half>(a, backward, grid, s) : launch_pair_of<__half, float>(a, backward, grid, s);
    *none = true;
    return cudaSuccess;
}
cudaError_t count_sms(int* sms) {
    static std::atomic<uint64_t> ready;
    return prepare_kernel((const void*)sums_kernel<1, 32>, 0, ready, sms);
}

}  // namespace

int norm_partial_rows(int T) { return T < kMostPartials ? T : kMostPartials; }

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    int sms = 0;
    cudaError_t err = count_sms(&sms);
    if (err != cudaSuccess) return err;
    bool none = a.T <= 2 * sms;
    if (!none) err = launch_rows(a, false, sms, s, &none);
    if (err != cudaSuccess || !none) return err;
    const bool f32 = a.x_type == MOE_F32 || a.y_type == MOE_F32;
    return !f32 && all_aligned(a, 8) ? rows_of<8>(a, s) : all_aligned(a, 4) ? rows_of<4>(a, s) : rows_of<1>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t err = count_sms(&sms);
    if (err != cudaSuccess) return err;
    int grid = std::min(norm_partial_rows(a.T), sms);
    if (a.T > 0) {
        const int most = (a.T + grid - 1) / grid;         // rows of a CTA: as many CTAs as that takes, no partial sums more
        grid = (a.T + most - 1) / most;
        bool none = false;
        err = launch_rows(a, true, grid, s, &none);
        if (none) {
            void* args[] = {const_cast<LayerNormArgs*>(&a)};
            err = launch_early((const void*)wide_backward_kernel, dim3(grid), 1024, 0, s, args);
        }
    }
    if (err != cudaSuccess || (!a.dgamma && !a.dbeta)) return err;
    const float* partial = a.partial;
    int H = a.H;
    float *dgamma = a.dgamma, *dbeta = a.dbeta;
    bool accumulate = a.accumulate;
    void* args[] = {&partial, &grid, &H, &dgamma, &dbeta, &accumulate};
    if (H % 4 == 0 && H >= 4096) return launch_early((const void*)sums_kernel<4, 16>, dim3((H + 127) / 128, 2), 512, 0, s, args);
    return launch_early((const void*)sums_kernel<1, 32>, dim3((H + 31) / 32, 2), 1024, 0, s, args);
}

}  // namespace moe
