// balance.cu -- the router's balance loss over T tokens in n_seqs sequences, its counts and its gradient.
//   p_te = softmax(l_t)_e, or sigmoid(l_te) / sum_j sigmoid(l_tj);  for sequence b of n_b counted tokens
//   f_be = E c_be / (k n_b)  (c_be: its tokens' pairs that name expert e),  P_be = sum_t p_te / n_b
//   loss = coef / B' sum_b sum_e f_be P_be   (B': sequences with a counted token)
//   d loss / d l_te = coef / (B' n_b) p_te (f_be - sum_j f_bj p_tj)   [sigmoid: times 1 - sigmoid(l_te)]
// Bound: bytes, the logits once and their gradient once.  The gradient needs f, which comes from the ids alone, and so does
// a token's share of the loss, coef / (B' n_b) sum_e f_be p_te, which the gradient needs as well: no sums of p by expert.
// So the ids are counted first (count_kernel), and one pass over the logits gives gradient and loss (pass_kernel; the CTA
// that ends last adds the others' shares of the loss).  A few tokens take one CTA that does both (small_kernel).
// The tokens are cut into even chunks, one for a CTA, whatever the sequences' lengths.  Chunk c of the tokens and sequence b
// that have tokens in common own row c + b of the partial counts: both only grow along the tokens, so no
// two such pairs share a row, and C chunks and B sequences need C + B rows.  Every sum has one order: the same bits each time
// (the only atomics are on whole numbers).
// f - 1 = (E c - k n) / (k n) takes the place of f in the gradient (the p sum to 1): nothing cancels where the load is balanced.
// No 64-bit floating point: its rate is a 64th of fp32's, and a handful of divisions took longer than the rest of a small call.
// Measured, loss, counts and gradient: 32 tokens of 128 experts, top 8, 5.0 us; 4096 of them, masked, 11.4 us (bytes alone 0.6): two launches,
// each with a chain of dependent reads; 32768 tokens of 256 experts in 16 sequences, sigmoid: 27.4 us (bytes alone 10.1), of
// which the counts take 8 and the pass 19, 58 % of its issue slots in use (an exponential and a reciprocal an element
// are among its instructions).  Loss and counts without the gradient: 9.6 and 22.9 us (bytes alone 0.3 and 5.1).
#include <algorithm>

#include "block_ops.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostChunks = 1024, kMostCounts = 128, kFewSeqs = 2;
constexpr float kInf = __builtin_huge_valf();
constexpr unsigned kAll = 0xffffffffu;

struct BalanceParams {
    BalanceArgs a;
    int chunks1, len1;           // count_kernel: CTAs, tokens of one
    int chunks2, len2;           // pass_kernel
    int row;                     // entries of a row of counts: E, the counted tokens, padding
    int32_t* counts;             // [chunks1 + n_seqs][row]
    float* losses;               // [chunks2] shares of the loss
    uint32_t* ticket;
    int32_t* used;               // [chunks1] sequences whose first counted token lies in the chunk
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
// Counted tokens of sequence b (a whole warp asks).
__device__ __forceinline__ int tokens_of(const BalanceParams& p, int b) {
    const int t0 = start_of(p.a, b), t1 = start_of(p.a, b + 1);
    if (!p.a.mask || t1 <= t0) return max(t1 - t0, 0);
    int n = 0;
    for (int c = t0 / p.len1 + (threadIdx.x & 31); c <= (t1 - 1) / p.len1; c += 32) n += p.counts[(int64_t)(c + b) * p.row + p.a.E];
    return __reduce_add_sync(kAll, n);
}
// Sequences with a counted token (a whole warp asks).
__device__ __forceinline__ int used_sequences(const BalanceParams& p) {
    int n = 0;
    for (int c = threadIdx.x & 31; c < p.chunks1; c += 32) n += p.used[c];
    return min(__reduce_add_sync(kAll, n), p.a.n_seqs);
}

// ---------------------------------------------------------------- counts
// The pairs of chunk c by sequence and expert.  hist: shared, [E + 1].
__device__ __forceinline__ void count_chunk(const BalanceParams& p, int c, int* hist) {
    const BalanceArgs& a = p.a;
    const int tid = threadIdx.x, t0 = c * p.len1, t1 = min(t0 + p.len1, a.T);
    bool bad = false;
    int used = 0;
    if (c == 0) {
        if (tid == 0) *p.ticket = 0;
        if (a.seq_offsets)
            for (int b = tid; b <= a.n_seqs; b += kThreads) {
                const int o = __ldg(a.seq_offsets + b);
                bad |= o < 0 || o > a.T || (b > 0 && __ldg(a.seq_offsets + b - 1) > o);
            }
    }
    for (int b = sequence_at(a, t0); b < a.n_seqs; ++b) {
        const int s0 = max(start_of(a, b), t0), s1 = min(start_of(a, b + 1), t1);
        if (start_of(a, b) >= t1) break;
        if (s1 <= s0) continue;
        bool before = false;                             // a token of the sequence counts in a chunk ahead
        if (!a.mask) before = start_of(a, b) < t0;
        else if (a.n_seqs > 1)                           // (one alone is used by as many chunks as it likes)
            for (int t = start_of(a, b) + tid; t - tid < t0 && !before; t += 4 * kThreads) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t + i * kThreads < t0) any |= a.mask[t + i * kThreads] != 0;
                before = __syncthreads_or(any);
            }
        for (int e = tid; e <= a.E; e += kThreads) hist[e] = 0;
        __syncthreads();
        if (a.mask)
            for (int t = s0 + tid; t < s1; t += kThreads)
                if (a.mask[t]) atomicAdd(&hist[a.E], 1);
#pragma unroll 4
        for (int i = s0 * a.k + tid; i < s1 * a.k; i += kThreads) {      // (T k <= 2^30)
            const int e = __ldg(a.ids + i);              // (beside the mask, not behind it)
            if (a.mask && !a.mask[(unsigned)i / (unsigned)a.k]) continue;
            if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
            else bad = true;
        }
        __syncthreads();
        used += !before && (!a.mask || hist[a.E] > 0);
        int32_t* out = p.counts + (int64_t)(c + b) * p.row;
        for (int e = tid; e <= a.E; e += kThreads) out[e] = hist[e];
        __syncthreads();
    }
    if (tid == 0) p.used[c] = used;
    if (__any_sync(kAll, bad) && (tid & 31) == 0 && a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
}
__global__ void __launch_bounds__(kThreads) count_kernel(const __grid_constant__ BalanceParams p) {
    extern __shared__ int hist[];
    wait_for_previous();
    allow_next();
    count_chunk(p, blockIdx.x, hist);
}

// ---------------------------------------------------------------- the pass over the logits
__device__ __forceinline__ float exp2_quick(float x) {    // relative error 2^-22; results below 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_quick(float x) {     // relative error 2^-23
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The sum over the CTA's threads, in one order (thread 0 has it).
__device__ __forceinline__ float cta_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    if (threadIdx.x == 0)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w];
    return v;
}
template <int EPL> constexpr int kResident = EPL <= 8 ? 2 : 1;     // CTAs an SM
// Chunk c of the tokens; the chunk's share of the loss (thread 0 has it).  A warp takes TOK tokens at a time; lane l holds
// experts (32 i + l) V + j of each, EPL in all.  fsm: shared, [E]; part: shared.
template <int EPL, int V, int TOK, bool SIGMOID>
__device__ __forceinline__ float pass_chunk(const BalanceParams& p, int c, float* fsm, float* part) {
    constexpr int NC = EPL / V;
    constexpr float kLog2e = 1.4426950408889634f, kBack = 2.3283064365386963e-10f;      // 2^-32
    const BalanceArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto expert = [&](int i) { return (i * 32 + lane) * V; };
    const bool logits = a.loss || a.dlogits;
    const int used = logits ? used_sequences(p) : 0;
    const float up = a.upstream ? __ldg(a.upstream) : 1.0f;
    const int t0 = c * p.len2, t1 = min(t0 + p.len2, a.T);
    float loss = 0.f;
    // gradient of the tokens that no sequence has, counts of the sequences without a token
    auto clear = [&](int g0, int g1) {
        if (!a.dlogits || a.accumulate) return;
        for (int t = g0 + warp; t < g1; t += kWarps)
            for (int e = lane; e < a.E; e += 32) a.dlogits[t * a.dstride + e] = 0.f;
    };
    clear(t0, min(start_of(a, 0), t1));
    clear(max(start_of(a, a.n_seqs), t0), t1);
    if (a.counts)
        for (int b = c; b < a.n_seqs; b += p.chunks2)
            if (start_of(a, b + 1) <= start_of(a, b))
                for (int e = tid; e < a.E; e += kThreads) a.counts[(int64_t)b * a.E + e] = 0;
    for (int b = sequence_at(a, t0); b < a.n_seqs; ++b) {
        const int b0 = start_of(a, b), b1 = start_of(a, b + 1), s0 = max(b0, t0), s1 = min(b1, t1);
        if (b0 >= t1) break;
        if (s1 <= s0) continue;
        // the mask of this warp's next 32 steps, a bit each: read step by step it held up the logits behind it (32768 tokens of 128
        // experts in 64 sequences 24.3 us, 18.9 without a mask)
        uint32_t seen[TOK];
        auto look = [&](int t) {
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const int at = t + o + lane * kWarps * TOK;
                seen[o] = __ballot_sync(kAll, at < s1 && (!a.mask || a.mask[at]));
            }
        };
        look(s0 + warp * TOK);
        int* cnt = reinterpret_cast<int*>(fsm);
        for (int e = tid; e < a.E; e += kThreads) cnt[e] = 0;
        __syncthreads();
        const int first = b0 / p.len1, rows = (b1 - 1) / p.len1 - first + 1;
        {
            // (four experts a lane, the rows dealt to the warps)
            constexpr int kFours = EPL <= 4 ? 1 : EPL / 4;
            int4 mine[kFours] = {};
#pragma unroll 4
            for (int i = warp; i < rows; i += kWarps)
#pragma unroll
                for (int j = 0; j < kFours; ++j)
                    if (4 * (lane + 32 * j) < a.E) {
                        const int4 v = *reinterpret_cast<const int4*>(p.counts + (int64_t)(first + i + b) * p.row + 4 * (lane + 32 * j));
                        mine[j].x += v.x; mine[j].y += v.y; mine[j].z += v.z; mine[j].w += v.w;
                    }
#pragma unroll
            for (int j = 0; j < kFours; ++j) {
                const int e = 4 * (lane + 32 * j);
                if (warp >= rows) continue;
                if (e < a.E) atomicAdd(&cnt[e], mine[j].x);
                if (e + 1 < a.E) atomicAdd(&cnt[e + 1], mine[j].y);
                if (e + 2 < a.E) atomicAdd(&cnt[e + 2], mine[j].z);
                if (e + 3 < a.E) atomicAdd(&cnt[e + 3], mine[j].w);
            }
        }
        const int n = tokens_of(p, b);
        const int64_t kn = (int64_t)a.k * n;
        const float inv_kn = n > 0 ? 1.0f / (float)kn : 0.f;
        __syncthreads();
        for (int e = tid; e < a.E; e += kThreads) {
            const int count = cnt[e];
            if (a.counts && b0 >= t0) a.counts[(int64_t)b * a.E + e] = count;     // (the chunk of its first token)
            fsm[e] = (float)((int64_t)a.E * count - kn) * inv_kn;
        }
        __syncthreads();
        const float weight = n > 0 && used > 0 ? a.coef / ((float)used * (float)n) : 0.f, scale = up * weight;
        float f[NC][V], shares = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) f[i][j] = expert(i) + j < a.E ? fsm[expert(i) + j] : 0.f;
        int step = 0;
        for (int tw = logits ? s0 + warp * TOK : s1; tw < s1; tw += kWarps * TOK, ++step) {
            if (step == 32) {
                look(tw);
                step = 0;
            }
            float l[TOK][NC][V], q[TOK][NC][V], m[TOK], sum[TOK], dot[TOK];
            bool live[TOK];
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const int t = tw + o;
                live[o] = (seen[o] >> step) & 1;
                const float* row = a.logits + t * a.stride;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
#pragma unroll
                    for (int j = 0; j < V; ++j) l[o][i][j] = -kInf;
                    if (live[o] && expert(i) < a.E) load_once<V>(row, MOE_F32, expert(i), l[o][i]);
                }
            }
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
                for (int o = 0; o < TOK; ++o) m[o] = fmaxf(m[o], __shfl_xor_sync(kAll, m[o], s));
            // q: p before its division, relative to the largest of them so that nothing underflows as a whole, and 2^32 times too
            // large so that none is lost that is not lost in p.  The 32 in the exponent rounds it to 2^-20: 6.6e-7 of each q at most,
            // where the instruction alone has 2.4e-7; gradients are off by 2e-7 in norm (fp32 exponentials without it: 7e-8 to 1.4e-7).
            // Adding it only to exponents below -64 would take two instructions more an element of a pass that the issue slots hold up.  A logit of -inf has p = 0, a token of nothing else no p at all.
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const float top = m[o] == -kInf ? 0.f : m[o];
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float v = l[o][i][j];
                        if constexpr (SIGMOID) {
                            // sigmoid = (v > 0 ? 1 : z) / (1 + z), 1 - sigmoid = (v > 0 ? z : 1) / (1 + z), z = e^-|v|
                            const float z = kBack * exp2_quick(fmaf(-kLog2e, fabsf(v), 32.0f)), one = rcp_quick(1.0f + z);
                            const bool up = v > 0.f;
                            q[o][i][j] = (up ? 1.0f : z) * one;
                            if (top >= 0.f) l[o][i][j] = (up ? z : 1.0f) * one;
                        } else {
                            q[o][i][j] = exp2_quick(fmaf(kLog2e, v - top, 32.0f));
                        }
                    }
                if (SIGMOID && top < 0.f) {
                    // negative logits alone (the token's whole warp): e^(v - max) in the place of z
#pragma unroll
                    for (int i = 0; i < NC; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float v = l[o][i][j], one = rcp_quick(1.0f + kBack * exp2_quick(fmaf(kLog2e, v, 32.0f)));
                            q[o][i][j] = exp2_quick(fmaf(kLog2e, v - top, 32.0f)) * one;
                            l[o][i][j] = one;
                        }
                }
                sum[o] = dot[o] = 0.f;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        sum[o] += q[o][i][j];
                        dot[o] = fmaf(q[o][i][j], f[i][j], dot[o]);
                    }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                for (int o = 0; o < TOK; ++o) {
                    sum[o] += __shfl_xor_sync(kAll, sum[o], s);
                    dot[o] += __shfl_xor_sync(kAll, dot[o], s);
                }
#pragma unroll
            for (int o = 0; o < TOK; ++o) {
                const int t = tw + o;
                const bool none = sum[o] == 0.f;
                const float inv = none ? 0.f : rcp_quick(sum[o]);
                dot[o] *= inv;
                if (!none) shares += 1.0f + dot[o];
                if (!a.dlogits || t >= s1 || (!live[o] && a.accumulate)) continue;
                float* row = a.dlogits + t * a.dstride;
                const float by = none ? 0.f : inv * scale;     // (0 whatever the upstream gradient: 0 * inf is no 0)
#pragma unroll
                for (int i = 0; i < NC; ++i) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        q[o][i][j] = (q[o][i][j] * by) * (f[i][j] - dot[o]);
                        if (SIGMOID) q[o][i][j] *= l[o][i][j];
                    }
                    if (expert(i) >= a.E) continue;
                    if (a.accumulate) {
                        float old[V];
                        load_once<V>(row, MOE_F32, expert(i), old);
#pragma unroll
                        for (int j = 0; j < V; ++j) q[o][i][j] += old[j];
                    }
                    store_row<V>(row, MOE_F32, expert(i), q[o][i]);
                }
            }
        }
        loss += shares * weight;
        __syncthreads();                                 // (fsm of the next sequence)
    }
    return a.loss ? cta_sum(lane == 0 ? loss : 0.f, part) : 0.f;
}
template <int EPL, int V, int TOK, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, kResident<EPL>) pass_kernel(const __grid_constant__ BalanceParams p) {
    extern __shared__ float fsm[];
    __shared__ float part[kWarps];
    __shared__ bool last;
    const BalanceArgs& a = p.a;
    const int tid = threadIdx.x;
    wait_for_previous();
    allow_next();
    float v = pass_chunk<EPL, V, TOK, SIGMOID>(p, blockIdx.x, fsm, part);
    if (!a.loss) return;
    if (tid == 0) {
        p.losses[blockIdx.x] = v;
        __threadfence();
        last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    v = 0.f;
    for (int i = tid; i < (int)gridDim.x; i += kThreads) v += __ldcg(p.losses + i);
    v = cta_sum(v, part);
    if (tid == 0) *a.loss = v;
}

// ---------------------------------------------------------------- a few tokens: one CTA, one launch
template <int EPL, int V, int TOK, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) small_kernel(const __grid_constant__ BalanceParams p) {
    extern __shared__ float fsm[];
    __shared__ float part[kWarps];
    wait_for_previous();
    allow_next();
    count_chunk(p, 0, reinterpret_cast<int*>(fsm));
    __syncthreads();
    const float v = pass_chunk<EPL, V, TOK, SIGMOID>(p, 0, fsm, part);
    if (p.a.loss && threadIdx.x == 0) *p.a.loss = v;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
// Chunks of the counts: about a thousand pairs each, and few enough that their rows are quickly added.
int count_chunks(int k, int T, int n_seqs) {
    const int64_t want = std::max<int64_t>((int64_t)T * k / 1024, n_seqs / 4);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, T), kMostCounts));
}
constexpr size_t kUsedAt = 256;                          // (in front of it: the ticket)
struct Layout {
    size_t counts, losses, total;
    int row;
};
Layout layout(int E, int n_seqs, int chunks1, int chunks2) {
    Layout l;
    l.row = (E + 4) & ~3;
    l.counts = kUsedAt + kMostCounts * 4;
    l.losses = align_up(l.counts + (size_t)(chunks1 + n_seqs) * l.row * 4, 256);
    l.total = align_up(l.losses + (size_t)chunks2 * 4, 256);
    return l;
}

template <int EPL, int V, int TOK, bool SIGMOID>
cudaError_t launch_pass(BalanceParams& p, bool small, cudaStream_t s) {
    static std::atomic<uint64_t> ready[2];
    int sms = 0;
    const void* fn = small ? (const void*)small_kernel<EPL, V, TOK, SIGMOID> : (const void*)pass_kernel<EPL, V, TOK, SIGMOID>;
    cudaError_t err = prepare_kernel(fn, 32 * EPL * 4 + 16, ready[small], &sms);
    if (err != cudaSuccess) return err;
    // even chunks, one for each CTA that runs at a time, of a token a warp or a sequence's tokens at least
    p.len2 = small ? std::max(p.a.T, 1)
                   : std::max(std::min(kWarps, ceil_div(p.a.T, p.a.n_seqs)), ceil_div(p.a.T, std::min(kResident<EPL> * sms, kMostChunks)));
    p.chunks2 = std::max(1, ceil_div(p.a.T, p.len2));
    void* args[] = {&p};
    return launch_early(fn, dim3(p.chunks2), kThreads, (size_t)p.a.E * 4 + 16, s, args);
}
template <bool SIGMOID>
cudaError_t launch_pass_of(BalanceParams& p, bool small, cudaStream_t s) {
    constexpr int kLess = SIGMOID ? 2 : 1;               // (its 1 - sigmoid takes registers)
    const BalanceArgs& a = p.a;
    const bool vec = a.E % 4 == 0 && (uintptr_t)a.logits % 16 == 0 && a.stride % 4 == 0 &&
                     (!a.dlogits || ((uintptr_t)a.dlogits % 16 == 0 && a.dstride % 4 == 0));
    if (vec)
        return a.E <= 128   ? launch_pass<4, 4, 4 / kLess, SIGMOID>(p, small, s)
               : a.E <= 256 ? launch_pass<8, 4, 2 / kLess, SIGMOID>(p, small, s)
               : a.E <= 512 ? launch_pass<16, 4, 1, SIGMOID>(p, small, s)
                            : launch_pass<32, 4, 1, SIGMOID>(p, small, s);
    return a.E <= 32    ? launch_pass<1, 1, 4, SIGMOID>(p, small, s)
           : a.E <= 128 ? launch_pass<4, 1, 4 / kLess, SIGMOID>(p, small, s)
           : a.E <= 256 ? launch_pass<8, 1, 2 / kLess, SIGMOID>(p, small, s)
           : a.E <= 512 ? launch_pass<16, 1, 1, SIGMOID>(p, small, s)
                        : launch_pass<32, 1, 1, SIGMOID>(p, small, s);
}

}  // namespace

size_t balance_ws_bytes(int E, int T, int n_seqs) { return layout(E, n_seqs, kMostCounts, std::max(1, std::min(T, kMostChunks))).total; }

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    int sms = 0;
    cudaError_t err = prepare_kernel((const void*)count_kernel, 8192, ready, &sms);
    if (err != cudaSuccess) return err;
    BalanceParams p{};
    p.a = a;
    // One launch where one CTA is not what takes the time: a few tokens in one or two sequences (it takes them one after another).
    // 128 experts, one launch / two: 64 tokens 5.7 / 6.9 us, in two sequences 8.5 / 8.7, in 8 23 / 9.2; 384 experts: 10 tokens
    // 5.0 / 7.4, 32 in two sequences 9.4 / 9.3, 64 8.5 / 7.6.
    const bool small = a.T <= 64 && a.T * a.E <= 16384 && std::min(a.T, a.n_seqs) <= kFewSeqs;
    p.len1 = small ? std::max(a.T, 1) : ceil_div(a.T, count_chunks(a.k, a.T, a.n_seqs));
    p.chunks1 = std::max(1, ceil_div(a.T, p.len1));
    const Layout l = layout(a.E, a.n_seqs, p.chunks1, 0);
    char* ws = static_cast<char*>(a.ws);
    p.row = l.row;
    p.ticket = reinterpret_cast<uint32_t*>(ws);
    p.used = reinterpret_cast<int32_t*>(ws + kUsedAt);
    p.counts = reinterpret_cast<int32_t*>(ws + l.counts);
    p.losses = reinterpret_cast<float*>(ws + l.losses);
    if (small) return a.sigmoid ? launch_pass_of<true>(p, true, s) : launch_pass_of<false>(p, true, s);
    void* args[] = {&p};
    err = launch_early((const void*)count_kernel, dim3(p.chunks1), kThreads, (size_t)(a.E + 1) * 4, s, args);
    if (err != cudaSuccess) return err;
    return a.sigmoid ? launch_pass_of<true>(p, false, s) : launch_pass_of<false>(p, false, s);
}

}  // namespace moe
