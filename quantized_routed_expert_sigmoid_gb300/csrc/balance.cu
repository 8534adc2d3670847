// balance.cu -- the router's balance loss over T tokens in n_seqs sequences, its counts and its gradient.
//   p_te = softmax(l_t)_e, or sigmoid(l_te) / sum_j sigmoid(l_tj);  for sequence b of n_b counted tokens
//   f_be = E c_be / (k n_b)  (c_be: its tokens' pairs that name expert e),  P_be = sum_t p_te / n_b
//   loss = coef / B' sum_b sum_e f_be P_be   (B': sequences with a counted token)
//   d loss / d l_te = coef / (B' n_b) p_te (f_be - sum_j f_bj p_tj)   [sigmoid: times 1 - sigmoid(l_te)]
// Bound: bytes, the logits once and their gradient once.  The gradient needs f, which comes from the ids alone, and not P:
// so the ids are counted first (count_kernel), one pass over the logits then gives the gradient and the partial
// sums of p (pass_kernel), and those are added up (finish_kernel).
// The tokens are cut into even chunks, one for a CTA, whatever the sequences' lengths.  Chunk c of the tokens and sequence b
// that have tokens in common own row c + b of the partial sums: both only grow along the tokens, so no
// two such pairs share a row, and C chunks and B sequences need C + B rows.  Every sum has one order: no atomics, the same
// bits each time.
// f - 1 = (E c - k n) / (k n) takes the place of f in the gradient (the p sum to 1): nothing cancels where the load is balanced.
#include <algorithm>

#include "block_ops.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostChunks = 1024;
constexpr float kInf = __builtin_huge_valf();

struct BalanceParams {
    BalanceArgs a;
    int chunks1, len1;           // count_kernel: CTAs, tokens of one
    int chunks2, len2;           // pass_kernel
    int row;                     // entries of a row of counts: E, the counted tokens, padding
    int32_t* counts;             // [chunks1 + n_seqs][row]
    float* sums;                 // [chunks2 + n_seqs][E]
    double* losses;              // [n_seqs][blocks of 32 experts]
    uint32_t* ticket;
};

// First token of sequence b (b <= n_seqs), clamped into 0..T.
__device__ __forceinline__ int start_of(const BalanceArgs& a, int b) {
    if (!a.seq_offsets) return b ? a.T : 0;
    return min(max(__ldg(a.seq_offsets + b), 0), a.T);
}
// The first sequence that ends behind token t (n_seqs: none).
__device__ __forceinline__ int sequence_at(const BalanceArgs& a, int t) {
    int lo = 0, hi = a.n_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start_of(a, mid + 1) > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}
// Calls f(chunk's row of the partial sums) for every chunk of `len` tokens that has tokens of sequence b.
template <typename F>
__device__ __forceinline__ void rows_of(const BalanceArgs& a, int b, int len, F f) {
    const int t0 = start_of(a, b), t1 = start_of(a, b + 1);
    if (t1 <= t0) return;
    for (int c = t0 / len; c <= (t1 - 1) / len; ++c) f(c + b);
}
// Counted tokens of sequence b.
__device__ __forceinline__ int tokens_of(const BalanceParams& p, int b) {
    if (!p.a.mask) return max(start_of(p.a, b + 1) - start_of(p.a, b), 0);
    int n = 0;
    rows_of(p.a, b, p.len1, [&](int r) { n += p.counts[(int64_t)r * p.row + p.a.E]; });
    return n;
}
// Sequences with a counted token (every thread of the CTA calls it).
__device__ __forceinline__ int used_sequences(const BalanceParams& p) {
    int n = 0;
    for (int b0 = 0; b0 < p.a.n_seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        n += __syncthreads_count(b < p.a.n_seqs && tokens_of(p, b) > 0);
    }
    return n;
}

// ---------------------------------------------------------------- counts
__global__ void __launch_bounds__(kThreads) count_kernel(const __grid_constant__ BalanceParams p) {
    extern __shared__ int hist[];                        // [E + 1]
    const BalanceArgs& a = p.a;
    const int tid = threadIdx.x;
    wait_for_previous();
    allow_next();
    bool bad = false;
    if (blockIdx.x == 0) {
        if (tid == 0) *p.ticket = 0;
        if (a.seq_offsets)
            for (int b = tid; b <= a.n_seqs; b += kThreads) {
                const int o = __ldg(a.seq_offsets + b);
                bad |= o < 0 || o > a.T || (b > 0 && __ldg(a.seq_offsets + b - 1) > o);
            }
    }
    const int c = blockIdx.x, t0 = c * p.len1, t1 = min(t0 + p.len1, a.T);
    for (int b = sequence_at(a, t0); b < a.n_seqs; ++b) {
        const int s0 = max(start_of(a, b), t0), s1 = min(start_of(a, b + 1), t1);
        if (start_of(a, b) >= t1) break;
        if (s1 <= s0) continue;
        for (int e = tid; e <= a.E; e += kThreads) hist[e] = 0;
        __syncthreads();
        if (a.mask)
            for (int t = s0 + tid; t < s1; t += kThreads)
                if (a.mask[t]) atomicAdd(&hist[a.E], 1);
        for (int64_t i = (int64_t)s0 * a.k + tid; i < (int64_t)s1 * a.k; i += kThreads) {
            if (a.mask && !a.mask[i / a.k]) continue;
            const int e = __ldg(a.ids + i);
            if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
            else bad = true;
        }
        __syncthreads();
        int32_t* out = p.counts + (int64_t)(c + b) * p.row;
        for (int e = tid; e <= a.E; e += kThreads) out[e] = hist[e];
        __syncthreads();
    }
    if (bad && a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
}

// ---------------------------------------------------------------- the pass over the logits
// A warp takes TOK tokens at a time; lane l holds experts (32 i + l) V + j of each, EPL in all.
template <int EPL, int V, int TOK>
__global__ void __launch_bounds__(kThreads) pass_kernel(const __grid_constant__ BalanceParams p) {
    extern __shared__ float fsm[];                       // [E] f - 1, then [warps][E] sums
    constexpr int NC = EPL / V;
    const BalanceArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto expert = [&](int i) { return (i * 32 + lane) * V; };
    wait_for_previous();
    allow_next();
    const int used = a.dlogits ? used_sequences(p) : 0;
    const float up = a.upstream ? __ldg(a.upstream) : 1.0f;
    const int c = blockIdx.x, t0 = c * p.len2, t1 = min(t0 + p.len2, a.T);
    // gradient of the tokens that no sequence has
    auto clear = [&](int g0, int g1) {
        if (!a.dlogits || a.accumulate) return;
        for (int64_t i = tid; i < (int64_t)(g1 - g0) * a.E; i += kThreads)
            a.dlogits[(g0 + i / a.E) * a.dstride + i % a.E] = 0.f;
    };
    clear(t0, min(start_of(a, 0), t1));
    clear(max(start_of(a, a.n_seqs), t0), t1);
    for (int b = sequence_at(a, t0); b < a.n_seqs; ++b) {
        const int s0 = max(start_of(a, b), t0), s1 = min(start_of(a, b + 1), t1);
        if (start_of(a, b) >= t1) break;
        if (s1 <= s0) continue;
        const int n = tokens_of(p, b);
        const int64_t kn = (int64_t)a.k * n;
        if (a.dlogits) {
            int* cnt = reinterpret_cast<int*>(fsm);
            for (int e = tid; e < a.E; e += kThreads) cnt[e] = 0;
            __syncthreads();
            const int first = start_of(a, b) / p.len1, rows = (start_of(a, b + 1) - 1) / p.len1 - first + 1;
            for (int i = warp; i < rows; i += kWarps)
                for (int e = lane; e < a.E; e += 32) atomicAdd(&cnt[e], p.counts[(int64_t)(first + i + b) * p.row + e]);
            __syncthreads();
            for (int e = tid; e < a.E; e += kThreads)
                fsm[e] = n > 0 ? (float)((double)((int64_t)a.E * cnt[e] - kn) / (double)kn) : 0.f;
            __syncthreads();
        }
        const float scale = n > 0 && used > 0 ? (float)((double)a.coef * up / ((double)used * n)) : 0.f;
        float acc[NC][V], f[NC][V];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc[i][j] = 0.f;
                f[i][j] = a.dlogits && expert(i) + j < a.E ? fsm[expert(i) + j] : 0.f;
            }
        for (int tw = s0 + warp * TOK; tw < s1; tw += kWarps * TOK) {
            float l[TOK][NC][V], q[TOK][NC][V];
            bool live[TOK];
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const int t = tw + o;
                live[o] = t < s1 && (!a.mask || a.mask[t]);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
#pragma unroll
                    for (int j = 0; j < V; ++j) l[o][i][j] = -kInf;
                    if (live[o] && expert(i) < a.E) load_once<V>(a.logits, MOE_F32, t * a.stride + expert(i), l[o][i]);
                }
            }
            float m[TOK], sum[TOK], dot[TOK];
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                m[o] = -kInf;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) m[o] = fmaxf(m[o], l[o][i][j]);
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                for (int o = 0; o < TOK; ++o) m[o] = fmaxf(m[o], __shfl_xor_sync(0xffffffffu, m[o], s));
            // q: p before its division, relative to the largest of them so that nothing underflows as a whole; a logit
            // of -inf has p = 0, a token of nothing else no p at all
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                sum[o] = dot[o] = 0.f;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float v = l[o][i][j];
                        if (a.sigmoid) {
                            const float z = expf(-fabsf(v)), one = 1.0f / (1.0f + z);
                            q[o][i][j] = v == -kInf ? 0.f : v > 0.f ? one : (m[o] < 0.f ? expf(v - m[o]) : z) * one;
                            l[o][i][j] = v > 0.f ? z * one : one;        // 1 - sigmoid
                        } else {
                            q[o][i][j] = v == -kInf ? 0.f : expf(v - m[o]);
                        }
                        sum[o] += q[o][i][j];
                        dot[o] = fmaf(q[o][i][j], f[i][j], dot[o]);
                    }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                for (int o = 0; o < TOK; ++o) {
                    sum[o] += __shfl_xor_sync(0xffffffffu, sum[o], s);
                    dot[o] += __shfl_xor_sync(0xffffffffu, dot[o], s);
                }
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const int t = tw + o;
                const float inv = sum[o] == 0.f ? 0.f : 1.0f / sum[o];
                dot[o] *= inv;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        q[o][i][j] *= inv;
                        acc[i][j] += q[o][i][j];         // (0 unless live)
                        q[o][i][j] *= scale * (f[i][j] - dot[o]);
                        if (a.sigmoid) q[o][i][j] *= l[o][i][j];
                    }
                    if (!a.dlogits || t >= s1 || expert(i) >= a.E) continue;
                    if (a.accumulate) {
                        if (!live[o]) continue;
                        float old[V];
                        load_once<V>(a.dlogits, MOE_F32, t * a.dstride + expert(i), old);
#pragma unroll
                        for (int j = 0; j < V; ++j) q[o][i][j] += old[j];
                    }
                    store_row<V>(a.dlogits, MOE_F32, t * a.dstride + expert(i), q[o][i]);
                }
            }
        }
        if (a.loss) {
            float* part = fsm + a.E;
            __syncthreads();                             // (the last sequence's sums have been read)
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (expert(i) + j < a.E) part[warp * a.E + expert(i) + j] = acc[i][j];
            __syncthreads();
            for (int e = tid; e < a.E; e += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += part[w * a.E + e];
                p.sums[(int64_t)(c + b) * a.E + e] = v;
            }
        }
        __syncthreads();                                 // (fsm and the sums of the next sequence)
    }
}

// ---------------------------------------------------------------- counts and loss of each sequence
// The sum of a double over the CTA's threads, in one order (thread 0 has it).
__device__ __forceinline__ double cta_sum(double v, double* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kWarps; ++w) v += part[w];
    return v;
}
// A CTA adds 32 experts' (blockIdx.x) partial rows of a sequence (blockIdx.y), the rows dealt to its warps.
__global__ void __launch_bounds__(kThreads) finish_kernel(const __grid_constant__ BalanceParams p) {
    __shared__ int cnt[kWarps][32];
    __shared__ float sum[kWarps][32];
    __shared__ double part[kWarps];
    __shared__ bool last;
    const BalanceArgs& a = p.a;
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, e = blockIdx.x * 32 + lane;
    wait_for_previous();
    allow_next();
    const int n = tokens_of(p, b), t0 = start_of(a, b), t1 = start_of(a, b + 1);
    int c = 0;
    float s = 0.f;
    if (e < a.E && t1 > t0) {
        for (int i = t0 / p.len1 + warp; i <= (t1 - 1) / p.len1; i += kWarps) c += p.counts[(int64_t)(i + b) * p.row + e];
        if (a.loss) {
#pragma unroll 4
            for (int i = t0 / p.len2 + warp; i <= (t1 - 1) / p.len2; i += kWarps) s += p.sums[(int64_t)(i + b) * a.E + e];
        }
    }
    cnt[warp][lane] = c;
    sum[warp][lane] = s;
    __syncthreads();
    double v = 0.0;
    if (warp == 0 && e < a.E) {
        c = 0;
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            c += cnt[w][lane];
            s += sum[w][lane];
        }
        if (a.counts) a.counts[(int64_t)b * a.E + e] = c;
        if (n > 0) v = (double)c * (double)s * a.E / ((double)a.k * n * n);
    }
    if (!a.loss) return;
    v = cta_sum(v, part);
    if (tid == 0) {
        p.losses[(int64_t)b * gridDim.x + blockIdx.x] = v;
        __threadfence();
        last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    const int used = used_sequences(p);
    v = 0.0;
    for (int64_t i = tid; i < (int64_t)gridDim.x * gridDim.y; i += kThreads) v += __ldcg(p.losses + i);
    v = cta_sum(v, part);
    if (tid == 0) *a.loss = used > 0 ? (float)(v * (double)a.coef / used) : 0.f;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
// Chunks of the counts: enough that a CTA has a few thousand pairs, few enough that their rows are quickly added.
int count_chunks(int k, int T, int n_seqs) {
    const int64_t want = std::max<int64_t>((int64_t)T * k / 4096, n_seqs / 4);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, T), 128));
}
struct Layout {
    size_t counts, sums, losses, total;
    int row;
};
Layout layout(int E, int n_seqs, int chunks1, int chunks2) {
    Layout l;
    l.row = (E + 4) & ~3;
    l.counts = 256;
    l.sums = align_up(l.counts + (size_t)(chunks1 + n_seqs) * l.row * 4, 256);
    l.losses = align_up(l.sums + (size_t)(chunks2 + n_seqs) * E * 4, 256);
    l.total = align_up(l.losses + (size_t)n_seqs * ((E + 31) / 32) * 8, 256);
    return l;
}

template <int EPL, int V, int TOK>
cudaError_t launch_pass(const BalanceParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    int sms = 0;
    const void* fn = (const void*)pass_kernel<EPL, V, TOK>;
    const int most = 32 * EPL * (1 + kWarps) * 4;
    cudaError_t err = prepare_kernel(fn, most, ready, &sms);
    if (err != cudaSuccess) return err;
    void* args[] = {const_cast<BalanceParams*>(&p)};
    return launch_early(fn, dim3(p.chunks2), kThreads, (size_t)p.a.E * (1 + kWarps) * 4, s, args);
}

}  // namespace

size_t balance_ws_bytes(int E, int T, int n_seqs) { return layout(E, n_seqs, 128, std::min(T, kMostChunks)).total; }

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    int sms = 0;
    cudaError_t err = prepare_kernel((const void*)count_kernel, 8192, ready, &sms);
    if (err != cudaSuccess) return err;
    BalanceParams p{};
    p.a = a;
    p.len1 = std::max(1, ceil_div(a.T, count_chunks(a.k, a.T, a.n_seqs)));
    p.chunks1 = std::max(1, ceil_div(a.T, p.len1));
    p.len2 = std::max(kWarps, ceil_div(a.T, std::min(2 * sms, kMostChunks)));
    p.chunks2 = ceil_div(a.T, p.len2);
    const Layout l = layout(a.E, a.n_seqs, p.chunks1, p.chunks2);
    char* ws = static_cast<char*>(a.ws);
    p.row = l.row;
    p.ticket = reinterpret_cast<uint32_t*>(ws);
    p.counts = reinterpret_cast<int32_t*>(ws + l.counts);
    p.sums = reinterpret_cast<float*>(ws + l.sums);
    p.losses = reinterpret_cast<double*>(ws + l.losses);
    void* args[] = {&p};
    err = launch_early((const void*)count_kernel, dim3(p.chunks1), kThreads, (size_t)(a.E + 1) * 4, s, args);
    if (err != cudaSuccess) return err;
    if (a.T > 0 && (a.loss || a.dlogits)) {
        const bool vec = a.E % 4 == 0 && (uintptr_t)a.logits % 16 == 0 && a.stride % 4 == 0 &&
                         (!a.dlogits || ((uintptr_t)a.dlogits % 16 == 0 && a.dstride % 4 == 0));
        if (vec)
            err = a.E <= 128   ? launch_pass<4, 4, 4>(p, s)
                  : a.E <= 256 ? launch_pass<8, 4, 2>(p, s)
                  : a.E <= 512 ? launch_pass<16, 4, 1>(p, s)
                               : launch_pass<32, 4, 1>(p, s);
        else
            err = a.E <= 32    ? launch_pass<1, 1, 4>(p, s)
                  : a.E <= 128 ? launch_pass<4, 1, 4>(p, s)
                  : a.E <= 256 ? launch_pass<8, 1, 2>(p, s)
                  : a.E <= 512 ? launch_pass<16, 1, 1>(p, s)
                               : launch_pass<32, 1, 1>(p, s);
        if (err != cudaSuccess) return err;
    }
    if (!a.loss && !a.counts) return cudaSuccess;
    return launch_early((const void*)finish_kernel, dim3((a.E + 31) / 32, a.n_seqs), kThreads, 0, s, args);
}

}  // namespace moe
