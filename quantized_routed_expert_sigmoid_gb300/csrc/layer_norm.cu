// layer_norm.cu -- layer norm, forward and backward:
//   m = mean x, r = 1 / sqrt(mean (x - m)^2 + eps), h = (x - m) r, y = h gamma + beta
//   g = dy gamma, dx = add + r (g - mean g - h mean(g h)), dgamma = sum_t dy h, dbeta = sum_t dy
// Bound: bytes.  A row is read once and stays in the registers of the threads that share it between its sums.  Threads
// take V neighbouring elements at a time, neighbouring threads neighbouring ones: 4 where an fp32 row is among
// them (16 bytes; eight in two halves would ask L2 for every 32-byte sector twice), 8 where all rows are 16-bit, one
// where rows are not aligned to that.
// A mean in fp32 is off by up to a few 2^-24 of the row's largest values, which is much of (x - m) where the
// row lies far from 0.  So the sum of (x - m) is taken along with that of its squares (no pass of its own) and the
// rest d = mean (x - m) is taken off: h = (x - m - d) r, the variance mean (x - m)^2 - d^2.  The backward pass, which gets
// the mean rounded to fp32, does the same.
#include <algorithm>

#include "block_ops.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
// Sums of v over the TPR threads of a row (all of them get the same bits).  part: [N][32] of the row's threads, not
// in use by a sum of theirs that some of them may still read.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* part, int group) {
    warp_sums(v);
    if constexpr (TPR > 32) {
        const int lane = threadIdx.x & 31, w = threadIdx.x % TPR / 32;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[i * 32 + w] = v[i];
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane < TPR / 32 ? part[i * 32 + lane] : 0.f;
        warp_sums(v);
    }
}

// ---------------------------------------------------------------- forward
// TPR threads a row, NC steps of V elements each.
template <int V, int TPR, int NC>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) layer_norm_kernel(const __grid_constant__ LayerNormArgs a) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kGroups = kThreads / TPR;
    __shared__ float part[2][kGroups][2 * 32];
    const int tid = threadIdx.x, group = tid / TPR, i0 = tid % TPR;
    wait_for_previous();
    allow_next();
    const int64_t t = (int64_t)blockIdx.x * kGroups + group;
    if (t >= a.T) return;                                // (a row's threads together: its barrier is their own)
    auto first = [&](int c) { return (c * TPR + i0) * V; };
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
    row_sums<TPR>(s, part[0][group], group);
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
    row_sums<TPR>(q, part[1][group], group);
    const float d = q[0] / (float)a.H;
    float var = q[1] / (float)a.H - d * d;
    if (var < 0.f) var = 0.f;                            // (a NaN stays)
    const float r = 1.0f / sqrtf(var + a.eps);
    if (i0 == 0) {
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
cudaError_t launch_forward(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kRows = kThreads / TPR;
    void* args[] = {const_cast<LayerNormArgs*>(&a)};
    return launch_early((const void*)layer_norm_kernel<V, TPR, NC>, dim3(((unsigned)a.T + kRows - 1) / kRows), kThreads, 0, s, args);
}
template <int V>
cudaError_t forward_of(const LayerNormArgs& a, cudaStream_t s) {
    if (a.H <= 256) return launch_forward<V, 32, 8 / V>(a, s);
    if (a.H <= 512) return launch_forward<V, 32, 16 / V>(a, s);
    if (a.H <= 1024) return launch_forward<V, 128, 8 / V>(a, s);
    if (a.H <= 2048) return launch_forward<V, 256, 8 / V>(a, s);
    if (a.H <= 4096) return launch_forward<V, 256, 16 / V>(a, s);
    if (a.H <= 8192) return launch_forward<V, 1024, 8 / V>(a, s);
    if (a.H <= 16384) return launch_forward<V, 1024, 16 / V>(a, s);
    return launch_forward<V, 1024, 32 / V>(a, s);
}

// ---------------------------------------------------------------- backward
// A CTA of GROUPS x TPR threads walks over the rows blockIdx.x + gridDim.x (group + GROUPS i); every thread keeps the
// sums for gamma and beta of its 8 channels in registers, joins them with the CTA's other groups in shared memory
// and writes one row of partial sums, which sums_kernel adds in a fixed order.
constexpr int kBackwardThreads = 512;

template <int V, int TPR>
__global__ void __launch_bounds__(TPR > kBackwardThreads ? TPR : kBackwardThreads)
    layer_norm_backward_kernel(const __grid_constant__ LayerNormArgs a) {
    constexpr int kThreads = TPR > kBackwardThreads ? TPR : kBackwardThreads, kGroups = kThreads / TPR, NC = 8 / V;
    __shared__ float part[2][kGroups][3 * 32];
    __shared__ float join[kGroups > 1 ? 2 * 8 * kThreads : 1];
    const int tid = threadIdx.x, group = tid / TPR, i0 = tid % TPR;
    auto first = [&](int c) { return (c * TPR + i0) * V; };
    wait_for_previous();
    allow_next();
    float gamma[NC][V], sg[NC][V], sb[NC][V];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < V; ++j) { gamma[c][j] = a.gamma ? 0.f : 1.f; sg[c][j] = sb[c][j] = 0.f; }
        if (a.gamma && first(c) < a.H) load_vec<V>(a.gamma, first(c), gamma[c]);
    }
    const float inv = 1.0f / (float)a.H;
    int turn = 0;
    for (int64_t t = blockIdx.x + (int64_t)gridDim.x * group; t < a.T; t += (int64_t)gridDim.x * kGroups, turn ^= 1) {
        float x[NC][V], dy[NC][V], q[3] = {0.f, 0.f, 0.f};
        const float m = __ldg(a.mean + t), r = __ldg(a.rstd + t);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int j = 0; j < V; ++j) { x[c][j] = m; dy[c][j] = 0.f; }
            if (first(c) < a.H) {
                load_once<V>(a.x, a.x_type, t * a.x_stride + first(c), x[c]);
                load_once<V>(a.y, a.y_type, t * a.y_stride + first(c), dy[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (first(c) >= a.H) continue;
                x[c][j] -= m;
                const float g = dy[c][j] * gamma[c][j];
                q[0] += g;
                q[1] = fmaf(g, x[c][j], q[1]);
                q[2] += x[c][j];
            }
        row_sums<TPR>(q, part[turn][group], group);
        const float d = q[2] * inv, m1 = q[0] * inv, m2 = (q[1] - d * q[0]) * r * inv;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (first(c) >= a.H) continue;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = (x[c][j] - d) * r;
                sg[c][j] = fmaf(dy[c][j], h, sg[c][j]);
                sb[c][j] += dy[c][j];
                o[j] = r * (dy[c][j] * gamma[c][j] - m1 - h * m2);
            }
            if (!a.dx) continue;
            if (a.add) {
                float v[V];
                load_once<V>(a.add, a.x_type, t * a.add_stride + first(c), v);
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += v[j];
            }
            store_row<V>(a.dx, a.x_type, t * a.dx_stride + first(c), o);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.H;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (first(c) < a.H) {
                    out[first(c) + j] = sg[c][j];
                    out[a.H + first(c) + j] = sb[c][j];
                }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                join[group * 8 * TPR + first(c) + j] = sg[c][j];
                join[8 * kThreads + group * 8 * TPR + first(c) + j] = sb[c][j];
            }
        __syncthreads();
        for (int i = tid; i < 2 * a.H; i += kThreads) {
            const int which = i >= a.H, h = i - which * a.H;
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) v += join[which * 8 * kThreads + g * 8 * TPR + h];
            out[i] = v;
        }
    }
}

// Rows of more than 8192 elements: they do not fit the registers beside the sums for gamma and beta, so a row is read
// twice (the second time from L1 and L2) and its share of those sums added to the CTA's row of partial sums in memory.
__global__ void __launch_bounds__(1024) layer_norm_backward_wide_kernel(const __grid_constant__ LayerNormArgs a) {
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
        for (int i = tid; i < a.H; i += 1024) {
            const float x = load1(a.x, a.x_type, t * a.x_stride + i) - m;
            const float g = load1(a.y, a.y_type, t * a.y_stride + i) * (a.gamma ? __ldg(a.gamma + i) : 1.f);
            q[0] += g;
            q[1] = fmaf(g, x, q[1]);
            q[2] += x;
        }
        row_sums<1024>(q, part[turn], 0);
        const float d = q[2] * inv, m1 = q[0] * inv, m2 = (q[1] - d * q[0]) * r * inv;
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

// dgamma, dbeta: the sums of the partial rows, 32 channels a CTA (blockIdx.y: gamma or beta).
__global__ void __launch_bounds__(512) sums_kernel(const float* partial, int rows, int H, float* dgamma, float* dbeta, bool accumulate) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? dbeta : dgamma;
    wait_for_previous();
    allow_next();
    if (!out) return;
    float v = 0.f;
    if (h < H)
#pragma unroll 4
        for (int i = w; i < rows; i += 16) v += partial[((int64_t)2 * i + blockIdx.y) * H + h];
    part[w][lane] = v;
    __syncthreads();
    if (w == 0 && h < H) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += part[i][lane];
        out[h] = accumulate ? out[h] + v : v;
    }
}

constexpr int kMostPartials = 512;

template <int V, int TPR>
cudaError_t launch_backward(const LayerNormArgs& a, int grid, cudaStream_t s) {
    constexpr int kThreads = TPR > kBackwardThreads ? TPR : kBackwardThreads;
    void* args[] = {const_cast<LayerNormArgs*>(&a)};
    return launch_early((const void*)layer_norm_backward_kernel<V, TPR>, dim3(grid), kThreads, 0, s, args);
}
template <int V>
cudaError_t backward_of(const LayerNormArgs& a, int grid, cudaStream_t s) {
    if (a.H <= 256) return launch_backward<V, 32>(a, grid, s);
    if (a.H <= 512) return launch_backward<V, 64>(a, grid, s);
    if (a.H <= 1024) return launch_backward<V, 128>(a, grid, s);
    if (a.H <= 2048) return launch_backward<V, 256>(a, grid, s);
    if (a.H <= 4096) return launch_backward<V, 512>(a, grid, s);
    return launch_backward<V, 1024>(a, grid, s);
}

// V elements of these rows can be read at once.
bool rows_of(const void* p, int type, int64_t stride, int v) {
    const int64_t bytes = (type == MOE_F32 ? 4 : 2) * v, whole = bytes > 16 ? 16 : bytes;
    return !p || ((uintptr_t)p % whole == 0 && stride * (type == MOE_F32 ? 4 : 2) % whole == 0);
}
int elements_of(const LayerNormArgs& a) {
    const bool f32 = a.x_type == MOE_F32 || a.y_type == MOE_F32;
    for (int v = f32 ? 4 : 8; v >= 4; v /= 2)
        if (a.H % v == 0 && rows_of(a.x, a.x_type, a.x_stride, v) && rows_of(a.y, a.y_type, a.y_stride, v) &&
            rows_of(a.add, a.x_type, a.add_stride, v) && rows_of(a.dx, a.x_type, a.dx_stride, v) &&
            rows_of(a.gamma, MOE_F32, 0, v) && rows_of(a.beta, MOE_F32, 0, v))
            return v;
    return 1;
}

}  // namespace

int norm_partial_rows(int T) { return T < kMostPartials ? T : kMostPartials; }

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    const int v = elements_of(a);
    return v == 8 ? forward_of<8>(a, s) : v == 4 ? forward_of<4>(a, s) : forward_of<1>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    int sms = 0;
    cudaError_t err = prepare_kernel((const void*)layer_norm_backward_wide_kernel, 0, ready, &sms);
    if (err != cudaSuccess) return err;
    const int grid = std::min(norm_partial_rows(a.T), sms * (a.H <= 4096 ? 2 : 1));
    if (a.T == 0) {
        // (no rows: sums of nothing)
    } else if (a.H > 8192) {
        void* args[] = {const_cast<LayerNormArgs*>(&a)};
        err = launch_early((const void*)layer_norm_backward_wide_kernel, dim3(grid), 1024, 0, s, args);
    } else {
        const int v = elements_of(a);
        err = v == 8 ? backward_of<8>(a, grid, s) : v == 4 ? backward_of<4>(a, grid, s) : backward_of<1>(a, grid, s);
    }
    if (err != cudaSuccess || (!a.dgamma && !a.dbeta)) return err;
    const float* partial = a.partial;
    int rows = grid, H = a.H;
    float *dgamma = a.dgamma, *dbeta = a.dbeta;
    bool accumulate = a.accumulate;
    void* args[] = {&partial, &rows, &H, &dgamma, &dbeta, &accumulate};
    return launch_early((const void*)sums_kernel, dim3((H + 31) / 32, 2), 512, 0, s, args);
}

}  // namespace moe
