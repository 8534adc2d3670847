// linear.cu -- a dense product with its epilogue on the 5th-generation tensor cores:
//   y[t, n] = res_scale * r[t, n] + scale * act(sum_c W[n, c] x[t, c] + bias[n])
// The weights are the M operand (a lane of TMEM holds one output channel, a column one row of x): a few rows of x
// then cost a few columns, and the bias is one register.  Everything behind the sum happens between TMEM and
// the one store of y, in fp32.  Two kernels; which one, and how a product is cut, is shape_of's model of their times:
// - split_kernel: tiles of 128 channels by up to 64 rows of x, one CTA each; where that leaves SMs idle, a cluster
//   of up to 8 CTAs splits the sum of a tile.  Each CTA sends the columns of its part to the CTA of the cluster that finishes
//   them (shared memory of the cluster, no workspace), which adds the parts in their order.
//   Bound: latency.  1 x 2048 -> 2048 with bias and residual, bf16: 5.2 us, 32 x 7168 -> 2048 with bias and GELU: 9.6 us, on
//   weights from HBM (their bytes alone: 1.2 and 4.4): 3 us are the launch, the first load and the closing code, the rest
//   is steps of the sum at 0.16 us each (8 and 19 of them a CTA).
// - pair_kernel: tiles of 256 channels by up to 256 rows, a pair of CTAs (cta_group::2) each, persistent, two accumulators: one
//   is read out while the next tile runs.  A weight is read from L2 once per 256 rows.
//   Bound: the matrix instructions (81 % of the pipe's time).  4096 x 2048 -> 7168, bf16 with bias and GELU: 67 us, 1.79 PFLOP/s
//   (1 less without an epilogue); 4096 x 7168 -> 2048 with bias and residual, fp32 outputs, sums in runs: 75 to 79 us, 1.6 PFLOP/s
//   (without residual 68.5).  Columns are dealt evenly to as few waves of tiles as
//   there can be: the last wave is what large products lose.
// The tensor cores cut a sum off after each instruction instead of rounding it, an error that grows with the
// sum's length; so long sums are made of runs (768 elements for fp32 outputs, 8192 for 16-bit ones), which the epilogue
// adds with rounding in its registers.
// Every wait is bounded; one that runs out is reported (MOE_ERR_TIMEOUT), the copies and MMAs in flight are waited for
// (bounded), TMEM is freed and the kernel returns.
#include <algorithm>

#include "block_ops.cuh"
#include "cluster_ptx.cuh"

namespace moe {
namespace {

constexpr int kStepK = 64;
constexpr int kRun32 = 12, kRun16 = 128;                 // steps of a run: fp32 outputs, 16-bit outputs
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;              // (a warp reads the TMEM lanes 32 (warp % 4)..)
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);

struct Epilogue {
    const void* bias;
    const void* r;
    void* y;
    int bias_type, r_type, y_type, act;
    int64_t r_stride, y_stride;
    float scale, res_scale;
    int T, N;
};

struct LinearParams {
    CUtensorMap tw;              // W: boxes of 64 x 128, or 64 x 64 of [K][N]
    CUtensorMap tx;              // x: boxes of 64 x (16 << box)
    Epilogue e;
    int nk, run;                 // nk: steps of the sum, run: of one run
    bool bf16;
    int cols;                    // columns of a tile (split: 16, 32 or 64; pairs: a multiple of 32)
    int box;                     // rows of a box of x: 16 << box
    int stages;
    bool vec;                    // four neighbouring channels of r and y can be read and written at once (split)
    int n_mb, n_tb;              // tiles along the channels and along the rows of x
    int32_t* status;
    uint64_t wait_ns;
    int stall;                   // test setting: the first wait of the MMA warp never completes
};

// ---------------------------------------------------------------- what follows the sum
// Powers of two and reciprocals by the one instruction (relative error of 2^-22 and 2^-23; subnormal results are 0).
__device__ __forceinline__ float exp2_quick(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_quick(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// e^-(w + more), w from 0 to 200, as value * back: 2^32 times too large where it would be subnormal.  `more` is what w lacks of the
// number that it stands for.  (Argument reduction in two parts, after Cody and Waite.)  The product with log2(e) is taken in two parts and the second one's power as 1 + x: relative error 2^-22 of
// the instruction and 2^-24.
__device__ __forceinline__ float exp_minus(float w, float more, float& back) {
    constexpr float kLog2e = 1.4426950408889634f, kRest = 1.9259629911266175e-8f;     // (log2(e) - kLog2e)
    const float p = w * -kLog2e, rest = fmaf(w, -kRest, fmaf(more, -kLog2e, fmaf(w, -kLog2e, -p)));
    const bool far = p < -64.0f;
    const float q = exp2_quick(far ? p + 32.0f : p);       // (exact: p has no bits below 2^-17 there)
    back = far ? 2.3283064365386963e-10f : 1.0f;
    return fmaf(q, rest * 0.69314718055994531f, q);
}
// FAST, for 16-bit outputs: relative error below 2e-5 (a 20th of half a step of fp16), most of it from the exponential's
// argument, rounded twice (2^-23 of up to 126 binary places) and from the polynomial below (5e-6).  Exponentials are taken
// 2^32 times too large, so that those of results that are subnormal are not, and are brought back by a product.
// GELU: Phi(-z) e^(z^2/2), z >= 0, the normal distribution's tail without its exponential, is a polynomial in
// t = 1 / (1 + 0.31 z) without constant term, fitted to it (least squares of the relative error, reweighted towards its
// largest values) on 0..14, where e^(-z^2/2) leaves fp32.
// For fp32 outputs: within 14 * 2^-24 (the exponential 5, polynomial and t 6, products 3; the polynomial, of degree 9 in
// 1 / (1 + 0.34 z), is off by 3e-8).  4096 x 2048 -> 7168 with silu, the
// tanh form and GELU: 86, 89 and 100 us, 70 without; 146, 162 and 204 with the library's functions, one value after another (their
// code is too long for a copy a value).
template <int ACT, bool FAST>
__device__ __forceinline__ float activate(float z) {
    constexpr float kBack = 2.3283064365386963e-10f;      // 2^-32
    if constexpr (ACT == MOE_ACT_RELU) {
        return z < 0.f ? 0.f : z;                         // (a NaN stays)
    } else if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU_TANH) {
        // z / (1 + e^-w), w = z or twice tanh's argument, from e^-|w|, which does not overflow
        const float w = ACT == MOE_ACT_SILU ? z : 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
        if constexpr (FAST) {
            const float q = kBack * exp2_quick(fmaf(-1.4426950408889634f, fabsf(w), 32.0f));
            return (w >= 0.f ? z : z * q) * rcp_quick(1.0f + q);
        } else {
            float back;
            const float q = exp_minus(fminf(fabsf(w), 200.0f), 0.f, back);
            return (w >= 0.f ? z : z * q * back) * rcp_quick(fmaf(q, back, 1.0f));
        }
    } else if constexpr (FAST) {
        const float t = rcp_quick(fmaf(0.31f, fabsf(z), 1.0f));
        float p = fmaf(t, kBack * -0.07392511516809464f, kBack * 0.18043823540210724f);
        p = fmaf(t, p, kBack * 0.01575886830687523f);
        p = fmaf(t, p, kBack * 0.13342174887657166f);
        p = fmaf(t, p, kBack * 0.12044348567724228f);
        p = fmaf(t, p, kBack * 0.12386047095060349f);
        const float q = t * p * exp2_quick(fmaf(z * z, -0.72134752044448170f, 32.0f));
        return z * (z >= 0.f ? 1.0f - q : q);
    } else {
        const float a = fminf(fabsf(z), 20.0f), s = a * a, t = rcp_quick(fmaf(0.34f, a, 1.0f));
        float back;
        const float e = exp_minus(0.5f * s, 0.5f * fmaf(a, a, -s), back);
        float p = fmaf(t, -0.026122288778424263f, 0.13950812816619873f);
        p = fmaf(t, p, -0.27315011620521545f);
        p = fmaf(t, p, 0.20220187306404114f);
        p = fmaf(t, p, -0.04473118856549263f);
        p = fmaf(t, p, 0.11536433547735214f);
        p = fmaf(t, p, 0.11519640684127808f);
        p = fmaf(t, p, 0.13611236214637756f);
        p = fmaf(t, p, 0.13562048971652985f);
        const float q = t * p * e;
        return z >= 0.f ? z * fmaf(q, -back, 1.0f) : z * q * back;
    }
}
template <bool FAST, int C>
__device__ __forceinline__ void activate_all(float (&v)[C], int act) {
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = f(v[i]);
    };
    switch (act) {
        case MOE_ACT_NONE: break;
        case MOE_ACT_RELU: each([](float z) { return activate<MOE_ACT_RELU, FAST>(z); }); break;
        case MOE_ACT_GELU: each([](float z) { return activate<MOE_ACT_GELU, FAST>(z); }); break;
        case MOE_ACT_GELU_TANH: each([](float z) { return activate<MOE_ACT_GELU_TANH, FAST>(z); }); break;
        default: each([](float z) { return activate<MOE_ACT_SILU, FAST>(z); }); break;
    }
}
template <int C>
__device__ __forceinline__ void activate_some(const Epilogue& e, float (&v)[C]) {
    if (e.y_type == MOE_F32) activate_all<false>(v, e.act);
    else activate_all<true>(v, e.act);
}

// The residual of channel n0 + lane for C rows of x from t0 on, of which n are there.  n0, t0 and n are the warp's, so that all but
// the lane's own offset is computed once for its lanes.  Asked for before the sums are there: the two latencies overlap.
template <int C, typename T>
__device__ __forceinline__ void load_channel(const Epilogue& e, float (&r)[C], int n0, int lane, int t0, int n) {
    const T* q = static_cast<const T*>(e.r) + ((int64_t)t0 * e.r_stride + n0);
    if (n0 + lane >= e.N) return;
#pragma unroll
    for (int i = 0; i < C; ++i, q += e.r_stride)
        if (i < n) r[i] = (float)q[lane];
}
template <int C>
__device__ __forceinline__ void load_residual(const Epilogue& e, float (&r)[C], int n0, int lane, int t0, int n) {
    if (!e.r) return;
    if (e.r_type == MOE_F32) load_channel<C, float>(e, r, n0, lane, t0, n);
    else if (e.r_type == MOE_BF16) load_channel<C, __nv_bfloat16>(e, r, n0, lane, t0, n);
    else load_channel<C, __half>(e, r, n0, lane, t0, n);
}
template <int C, typename T>
__device__ __forceinline__ void store_channel(const Epilogue& e, const float (&v)[C], int n0, int lane, int t0, int n) {
    T* q = static_cast<T*>(e.y) + ((int64_t)t0 * e.y_stride + n0);
    if (n0 + lane >= e.N) return;
    if (n >= C) {
#pragma unroll
        for (int i = 0; i < C; ++i, q += e.y_stride) q[lane] = to_out<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i, q += e.y_stride)
            if (i < n) q[lane] = to_out<T>(v[i]);
    }
}
// The same values, finished and stored.
template <int C>
__device__ __forceinline__ void finish(const Epilogue& e, float bias, float (&v)[C], const float (&r)[C], int n0, int lane, int t0, int n) {
    if (e.act == MOE_ACT_NONE) {
        const float b = bias * e.scale;
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = fmaf(v[i], e.scale, b);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] += bias;
        activate_some(e, v);
        if (e.scale != 1.0f)
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] *= e.scale;
    }
    if (e.r)
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = fmaf(e.res_scale, r[i], v[i]);
    if (e.y_type == MOE_F32) store_channel<C, float>(e, v, n0, lane, t0, n);
    else if (e.y_type == MOE_BF16) store_channel<C, __nv_bfloat16>(e, v, n0, lane, t0, n);
    else store_channel<C, __half>(e, v, n0, lane, t0, n);
}
__device__ __forceinline__ float bias_at(const Epilogue& e, int row) {
    return e.bias && row < e.N ? load1(e.bias, e.bias_type, row) : 0.f;
}

__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void prefetch_l2(const void* p, int type, int64_t i) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + i * (type == MOE_F32 ? 4 : 2)));
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

// ---------------------------------------------------------------- one CTA a tile, the sum split over a cluster
// A lane's four channels of the 128 of a tile: neighbours where r and y can be read and written 4 at a time, else each 32nd.
__device__ __forceinline__ int channel(int lane, int i, bool vec) { return vec ? 4 * lane + i : lane + 32 * i; }
__device__ __forceinline__ void load_residual4(const LinearParams& p, float (&r)[4], int n0, int lane, int64_t t) {
    const Epilogue& e = p.e;
    const int64_t at = t * e.r_stride + n0;
    if (p.vec) {
        if (n0 + 4 * lane < e.N) load_once<4>(e.r, e.r_type, at + 4 * lane, r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + lane + 32 * i < e.N) r[i] = load1(e.r, e.r_type, at + lane + 32 * i);
    }
}
__device__ __forceinline__ void finish4(const LinearParams& p, const float (&bias)[4], float (&v)[4], const float (&r)[4], int n0,
                                        int lane, int64_t t, bool store) {
    const Epilogue& e = p.e;
    if (e.act == MOE_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i], e.scale, bias[i] * e.scale);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += bias[i];
        activate_some(e, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= e.scale;
    }
    if (e.r)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(e.res_scale, r[i], v[i]);
    const int64_t at = t * e.y_stride + n0;
    if (p.vec) {
        if (store && n0 + 4 * lane < e.N) store_row<4>(e.y, e.y_type, at + 4 * lane, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (store && n0 + lane + 32 * i < e.N) store_value(e.y, e.y_type, at + lane + 32 * i, v[i]);
    }
}

constexpr int kABytes = 128 * 128;                       // a step's weights
// Steps of the sum that a stage of a ring holds.  A stage costs about 300 clocks of waiting, issuing and committing whatever it
// holds (without loads and with one instruction a step still 335 of 435 clocks a step), more than the matrix instructions of a step
// of up to 128 columns take.
constexpr int kPer = 2;
constexpr int kMaxStages = 6;

template <bool IN_OUT, int COLS>
__global__ void __launch_bounds__(kThreads, COLS <= 32 ? 2 : 1) split_kernel(const __grid_constant__ LinearParams p) {
    constexpr int kStep = kABytes + COLS * 128, kStage = kPer * kStep, kHalf = COLS / 2;
    constexpr uint32_t kTmem = 2 * COLS < 32 ? 32 : 2 * COLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], accf[2], accr[2], drain, never, parts_here;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, issued;
    volatile int* abort_flag = &abort_word;
    // parts: [CTA of the cluster][columns that this one finishes][128 channels], as the others send them.  What this CTA sends,
    // [column][128 channels], takes the place of the stages, which are used up by then (alone, it finishes that itself).
    float* parts = reinterpret_cast<float*>(smem + max(p.stages * kStage, COLS * 512));
    float* sent = reinterpret_cast<float*>(smem);

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int rank = uniform((int)cta_rank());
    uint32_t splits;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    splits = uniform(splits);
    const int mb = blockIdx.x / splits, tok0 = blockIdx.y * COLS;
    const int k0 = (int)((int64_t)p.nk * rank / splits), k1 = (int)((int64_t)p.nk * (rank + 1) / splits);
    const int n_runs = (k1 - k0 + p.run - 1) / p.run;
    const int most = (COLS + (int)splits - 1) / (int)splits;           // columns that a CTA of the cluster finishes, at most
    const int own = max(0, min(most, COLS - rank * most));
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&accf[i], 1); mbar_init(&accr[i], kEpiWarps); }
        mbar_init(&drain, 1);
        mbar_init(&never, 1);
        mbar_init(&parts_here, 1);
        abort_word = 0;
        issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (splits > 1)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&parts_here)), "r"(own * (int)splits * 512)
                         : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)), "n"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 64) prefetch_map(&p.tw);
    if (tid == 96) prefetch_map(&p.tx);
    __syncwarp();
    tc_before();
    __syncthreads();
    cluster_arrive();                                    // (the cluster's CTAs run: waited for before the first part is sent)
    tc_after();
    const uint32_t tmem = tmem_slot;
    wait_for_previous();
    allow_next();

    if (warp == 0) {
        // ======================= loads =======================
        // (the whole warp keeps step, so that what one lane issues lies in uniform registers)
        const uint32_t stage0 = su32(smem), full0 = su32(full);
        const CUtensorMap* xmap = &p.tx;
        int g = 0, s = 0;
        uint32_t ph = 1;
        for (int kb = k0; kb < k1; kb += kPer, ++g) {
            if (!wait_warp(&empty[s], ph, abort_flag, p.wait_ns)) break;
            const uint32_t bar = full0 + 8 * s, bytes = (uint32_t)min(kPer, k1 - kb) * kStep;
            if (elect_one()) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    if (kb + u >= k1) break;
                    const uint32_t a = stage0 + s * kStage + u * kStep;
                    const int c = (kb + u) * kStepK;
                    if constexpr (IN_OUT) {
                        tma_load(a, &p.tw, mb * 128, c, bar);
                        tma_load(a + 8192, &p.tw, mb * 128 + 64, c, bar);
                    } else {
                        tma_load(a, &p.tw, c, mb * 128, bar);
                    }
                    tma_load(a + kABytes, xmap, c, tok0, bar);
                }
            }
            __syncwarp();
            if (++s == p.stages) { s = 0; ph ^= 1; }
        }
        if (lane == 0) issued = g;
    } else if (warp == 1) {
        // ======================= MMA issue =======================
        const uint32_t idesc = uniform(idesc_mma(128, COLS, p.bf16) | (IN_OUT ? 1u << 15 : 0u));
        const uint32_t a0 = su32(smem);
        const uint64_t da0 = IN_OUT ? sdesc_mn(a0) : sdesc(a0), db0 = sdesc(a0 + kABytes);
        constexpr uint32_t kAdvA = (IN_OUT ? 2048 : 32) >> 4, kAdvB = 32 >> 4;
        int s = 0, j = 0;
        uint32_t ph = 0;
        bool ok = true, any = false;
        for (int r0 = k0; ok && r0 < k1; r0 += p.run, ++j) {
            const int b = j & 1, r1 = min(r0 + p.run, k1);
            if (j >= 2 && !wait_warp(&accr[b], ((j >> 1) - 1) & 1, abort_flag, p.wait_ns)) break;
            tc_after();
            const uint32_t acc = uniform(tmem + (uint32_t)b * COLS);
            for (int kb = r0; kb < r1; kb += kPer) {
                const bool stalled = p.stall && !any;    // (test setting)
                if (!wait_warp(stalled ? &never : &full[s], stalled ? 0u : ph, abort_flag, p.wait_ns)) { ok = false; break; }
                tc_after();
                const uint32_t adv = (uint32_t)s * (kStage >> 4);
                const uint64_t da = da0 + adv, db = db0 + adv;
                if (elect_one()) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u) {
                        if (kb + u >= r1) break;
#pragma unroll
                        for (int kk = 0; kk < kStepK / 16; ++kk)
                            mma_f16(acc, da + u * (kStep >> 4) + kk * kAdvA, db + u * (kStep >> 4) + kk * kAdvB, idesc, u > 0 || kk > 0 || kb > r0);
                    }
                    mma_commit(&empty[s]);
                    if (kb + kPer >= r1) mma_commit(&accf[b]);
                }
                __syncwarp();
                any = true;
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
        }
        if (any) {                                       // every MMA issued has completed before TMEM is freed
            if (elect_one()) mma_commit(&drain);
            __syncwarp();
            drain_wait(&drain, 0, p.wait_ns);
        }
    }
    __syncwarp();
    cluster_wait();
    if (warp >= kEpiWarp0) {
        // ======================= epilogue =======================
        const int q = warp & 3, side = (warp - kEpiWarp0) >> 2, w = warp - kEpiWarp0, n0 = mb * 128, t0 = tok0 + rank * most;
        float bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = bias_at(p.e, n0 + channel(lane, i, p.vec));
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + side * kHalf;
        const float* at = splits > 1 ? parts : sent;
        float res[2][4] = {};                            // of columns c and c + 8
        if (p.e.r)                                       // the residual into L2, a line of 32 channels a lane
            for (int c = w + (lane >> 2) * kEpiWarps; c < own; c += 8 * kEpiWarps)
                if (t0 + c < p.e.T && n0 + 32 * (lane & 3) < p.e.N)
                    prefetch_l2(p.e.r, p.e.r_type, (t0 + c) * p.e.r_stride + n0 + 32 * (lane & 3));
        bool ok = true;
        // Turn 0 runs the code that ends the kernel on no rows at all, while the first weights are on their way: read
        // from memory at its first use, it takes longer than what it does (2.5 us for one row of x, of 12).
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            const int end = turn ? min(t0 + own, p.e.T) : t0;
            if (turn) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (p.e.r && t0 + w + h * kEpiWarps < end) load_residual4(p, res[h], n0, lane, t0 + w + h * kEpiWarps);
                // the sums, run by run
                float sum[kHalf];
                for (int j = 0; j < n_runs; ++j) {
                    const int b = j & 1;
                    ok = wait_warp(&accf[b], (j >> 1) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_after();
#pragma unroll
                    for (int c = 0; c < kHalf; c += 8) {
                        uint32_t v[8];
                        tmem_ld8(lanes + b * COLS + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sum[c + i] = j ? __fadd_rn(sum[c + i], __uint_as_float(v[i])) : __uint_as_float(v[i]);
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&accr[b]);
                }
                if (ok) {
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) sent[(side * kHalf + c) * 128 + q * 32 + lane] = sum[c];
                }
                if (splits > 1) fence_async_smem();
                ok = all_of(1, 32 * kEpiWarps, ok);
                if (splits > 1) {
                    if (ok && warp == kEpiWarp0 && lane < (int)splits) {
                        // columns lane * most .. to CTA `lane`, where this CTA's place is `rank`
                        const uint32_t bytes = (uint32_t)max(0, min(most, COLS - lane * most)) * 512;
                        if (bytes)
                            asm volatile(
                                "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                    in_cta(su32(parts) + rank * bytes, lane)),
                                "r"(su32(sent) + lane * most * 512), "r"(bytes), "r"(in_cta(su32(&parts_here), lane))
                                : "memory");
                    }
                    __syncwarp();
                    ok = ok && wait_warp(&parts_here, 0, abort_flag, p.wait_ns);
                    if (!ok && lane == 0) drain_wait(&parts_here, 0, p.wait_ns);
                    __syncwarp();
                    cluster_arrive();                    // (what the others sent here has arrived, or this CTA has given up)
                }
                if (!ok) break;
            }
#pragma unroll 1
            for (int c = w; !turn || t0 + c < end; c += 2 * kEpiWarps) {
                float v[2][4] = {}, r[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[h][i] = res[h][i];
                    const int next = t0 + c + (2 + h) * kEpiWarps;
                    if (p.e.r && next < end) load_residual4(p, res[h], n0, lane, next);
                }
                const float* from = at + c * 128;
                if (turn)
                    for (int s = 0; s < (int)splits; ++s, from += own * 128)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h && t0 + c + kEpiWarps >= end) break;
                            const float* f = from + h * kEpiWarps * 128;
                            if (p.vec) {
                                const float4 u = *reinterpret_cast<const float4*>(f + 4 * lane);
                                v[h][0] += u.x; v[h][1] += u.y; v[h][2] += u.z; v[h][3] += u.w;
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i) v[h][i] += f[lane + 32 * i];
                            }
                        }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    finish4(p, bias, v[h], r[h], n0, lane, t0 + c + h * kEpiWarps, turn && t0 + c + h * kEpiWarps < end);
                if (!turn) break;
            }
        }
    } else if (splits > 1) {
        cluster_arrive();
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (tid == 0 && *abort_flag) {
        // copies in flight: wait, within the limit, for their bytes
        for (int g = max(0, issued - p.stages); g < issued; ++g) drain_wait(&full[g % p.stages], (g / p.stages) & 1, p.wait_ns);
        if (p.status) atomicCAS(p.status, (int)MOE_OK, (int)MOE_ERR_TIMEOUT);
    }
    __syncwarp();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmem) : "memory");
    __syncwarp();
    if (splits > 1) cluster_wait();                      // (what this CTA sent is no longer read)
}

// ---------------------------------------------------------------- a pair of CTAs a tile
// Steps a stage, stages and bytes of one: wide tiles (more than 128 columns, which the matrix instructions bound) and narrow ones.
constexpr int kPairCols = 256;
template <bool WIDE> constexpr int kPairPer = WIDE ? 1 : kPer;
template <bool WIDE> constexpr int kPairStages = WIDE ? 6 : 4;
template <bool WIDE> constexpr int kPairStep = kABytes + (WIDE ? 128 : 64) * 128;
constexpr uint32_t kPairTmem = 512;
constexpr int kPairEpi0 = 2;
// Epilogue warps: 16, or 8 that have the registers for the sums of 128 columns each.
template <bool RUNS> constexpr int kPairEpiWarps = RUNS ? 8 : 16;
template <bool RUNS> constexpr int kPairThreads = 32 * (kPairEpi0 + kPairEpiWarps<RUNS>);

template <bool IN_OUT, bool RUNS, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads<RUNS>, 1) pair_kernel(const __grid_constant__ LinearParams p) {
    constexpr int kStages = kPairStages<WIDE>, kP = kPairPer<WIDE>, kStep = kPairStep<WIDE>, kStage = kP * kStep;
    using Ring = RingOf<kStages>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kStages], empty[kStages], accf[2], accr[2], drain, never;   // full, accr: the first CTA's
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, issued;
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = uniform((int)threadIdx.x >> 5), lane = tid & 31;
    const uint32_t cta = uniform(cta_rank());
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 2); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&accf[i], 1); mbar_init(&accr[i], 2 * kPairEpiWarps<RUNS>); }
        mbar_init(&drain, 1);
        mbar_init(&never, 1);
        abort_word = 0;
        issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tw);
        prefetch_map(&p.tx);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)), "n"(kPairTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    cluster_sync();
    tc_after();
    const uint32_t tmem = tmem_slot;
    wait_for_previous();
    allow_next();
    const int n_pairs = gridDim.x >> 1, first = blockIdx.x >> 1, n_tiles = p.n_mb * p.n_tb;
    const int nh = p.cols >> 1;                          // this CTA's columns

    if (warp == 0) {
        // ======================= loads =======================
        const uint32_t full0 = in_leader(su32(full)), stage0 = su32(smem);
        const uint32_t step_bytes = kABytes + (2048u << p.box);
        int g = 0;
        Ring ring;
        bool ok = true;
        for (int t = first; ok && t < n_tiles; t += n_pairs) {
            const int tb = t / p.n_mb, mb = t - tb * p.n_mb;
            const int c0 = uniform(tb * p.cols + (int)cta * nh), r0 = uniform(mb * 256 + (int)cta * 128);
            for (int kb = 0; kb < p.nk; kb += kP, ++g, ring.next()) {
                if (!wait_warp(&empty[ring.s], ring.ph ^ 1, abort_flag, p.wait_ns)) { ok = false; break; }
                const uint32_t bar = full0 + 8 * ring.s, bytes = (uint32_t)min(kP, p.nk - kb) * step_bytes;
                if (elect_one()) {
                    arrive_tx_cluster(bar, bytes);
#pragma unroll
                    for (int u = 0; u < kP; ++u) {
                        if (kb + u >= p.nk) break;
                        const uint32_t a = stage0 + ring.s * kStage + u * kStep;
                        const int c = (kb + u) * kStepK;
                        if constexpr (IN_OUT) {
                            tma_2d(a, &p.tw, r0, c, bar);
                            tma_2d(a + 8192, &p.tw, r0 + 64, c, bar);
                        } else {
                            tma_2d(a, &p.tw, c, r0, bar);
                        }
                        tma_2d(a + kABytes, &p.tx, c, c0, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) issued = g;
        // the last steps' arrivals on this CTA's barriers have landed before it may leave
        if (g < kStages) { ring.s = 0; ring.ph = 1; }
        for (int i = 0; ok && i < min(g, kStages); ++i, ring.next())
            ok = wait_warp(&empty[ring.s], ring.ph ^ 1, abort_flag, p.wait_ns);
    } else if (warp == 1) {
        // ======================= MMA issue (in the first CTA) =======================
        if (cta == 0) {
            const uint32_t a0 = su32(smem);
            const uint64_t da0 = IN_OUT ? sdesc_mn(a0) : sdesc(a0), db0 = sdesc(a0 + kABytes);
            constexpr uint32_t kAdvA = (IN_OUT ? 2048 : 32) >> 4, kAdvB = 32 >> 4;
            const uint32_t idesc = uniform(idesc_mma(256, p.cols, p.bf16) | (IN_OUT ? 1u << 15 : 0u));
            Ring ring;
            int j = 0;
            bool ok = true, any = false;
            for (int t = first; ok && t < n_tiles; t += n_pairs) {
                for (int kb = 0, start = 0, b = 0; kb < p.nk; kb += kP, ring.next()) {
                    if (kb == start) {                   // the first step of a run
                        b = j & 1;
                        if (j >= 2 && !wait_warp(&accr[b], ((j >> 1) - 1) & 1, abort_flag, p.wait_ns)) { ok = false; break; }
                        tc_after();
                    }
                    const uint32_t acc = uniform(tmem + (uint32_t)b * kPairCols);
                    const bool last_step = kb + kP >= p.nk || kb + kP - start >= p.run;
                    const bool stalled = p.stall && !any;            // (test setting)
                    if (!wait_warp(stalled ? &never : &full[ring.s], stalled ? 0u : ring.ph, abort_flag, p.wait_ns)) { ok = false; break; }
                    tc_after();
                    const uint32_t adv = (uint32_t)ring.s * (kStage >> 4);
                    const uint64_t da = da0 + adv, db = db0 + adv;
                    if (elect_one()) {
#pragma unroll
                        for (int u = 0; u < kP; ++u) {
                            if (kb + u >= p.nk) break;
#pragma unroll
                            for (int kk = 0; kk < kStepK / 16; ++kk)
                                mma_pair(acc, da + u * (kStep >> 4) + kk * kAdvA, db + u * (kStep >> 4) + kk * kAdvB, idesc,
                                         u > 0 || kk > 0 || kb > start);
                        }
                        commit_pair(&empty[ring.s]);
                        if (last_step) commit_pair(&accf[b]);
                    }
                    __syncwarp();
                    if (last_step) { start = kb + kP; ++j; }
                    any = true;
                }
            }
            if (any) {                                   // every MMA issued has completed before TMEM is freed
                if (elect_one())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(&drain))
                                 : "memory");
                __syncwarp();
                drain_wait(&drain, 0, p.wait_ns);
            }
        }
    } else {
        // ======================= epilogue: lanes 32 q.. of TMEM, columns 16 side .. of every kEvery =======================
        constexpr int kSides = kPairEpiWarps<RUNS> / 4, kEvery = 16 * kSides;
        const int q = uniform(warp & 3), side = uniform((warp - kPairEpi0) >> 2);
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + 16 * side, accr0 = in_leader(su32(accr));
        auto release = [&](int b) {
            tc_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(accr0 + 8 * b);
        };
        int j = 0;
        bool ok = true;
        for (int t = first; ok && t < n_tiles; t += n_pairs) {
            const int tb = t / p.n_mb, mb = t - tb * p.n_mb;
            const int n0 = uniform(mb * 256 + (int)cta * 128 + q * 32), tok0 = uniform(tb * p.cols + 16 * side);
            const int n = uniform(min(tb * p.cols + p.cols, p.e.T)) - tok0;      // (columns c < n are there)
            const float bias = bias_at(p.e, n0 + lane);
            if constexpr (RUNS) {
                float sum[kPairCols / kSides];
                for (int k0 = 0; k0 < p.nk; k0 += p.run, ++j) {
                    const int b = j & 1;
                    ok = wait_warp(&accf[b], (j >> 1) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_after();
                    // the tile's residual into L2 while the last two runs go on (a line of a row of x a lane)
                    if (p.e.r && k0 + 2 * p.run >= p.nk && k0 + p.run < p.nk && n0 < p.e.N)
                        for (int c = (lane & 15) + kEvery * (lane >> 4); c < n; c += 2 * kEvery)
                            prefetch_l2(p.e.r, p.e.r_type, (tok0 + c) * p.e.r_stride + n0);
#pragma unroll
                    for (int i = 0; i < kPairCols / kSides; i += 16)
                        if (i * kSides < n) {
                            uint32_t v[16];
                            tmem_ld16(lanes + b * kPairCols + i * kSides, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                sum[i + e] = k0 ? __fadd_rn(sum[i + e], __uint_as_float(v[e])) : __uint_as_float(v[e]);
                        }
                    release(b);
                }
                if (!ok) break;
#pragma unroll 1
                for (int c = 0; c < n; c += kEvery) {                // (one copy of the code: the sums pass by)
                    float v[16], r[16];
                    load_residual<16>(p.e, r, n0, lane, tok0 + c, n - c);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = sum[e];
#pragma unroll
                    for (int e = 0; e + 16 < kPairCols / kSides; ++e) sum[e] = sum[e + 16];
                    finish<16>(p.e, bias, v, r, n0, lane, tok0 + c, n - c);
                }
            } else {
                const int b = j & 1;
                float res[16];
                load_residual<16>(p.e, res, n0, lane, tok0, n);
                ok = wait_warp(&accf[b], (j >> 1) & 1, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_after();
                uint32_t u[16];
                if (n > 0) tmem_ld16(lanes + b * kPairCols, u);
                for (int c = 0; c < n; c += kEvery) {
                    float v[16], r[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = res[i];
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
                    if (c + kEvery < n) {
                        tmem_ld16(lanes + b * kPairCols + c + kEvery, u);
                        load_residual<16>(p.e, res, n0, lane, tok0 + c + kEvery, n - c - kEvery);
                    } else {
                        release(b);                      // (everything is read)
                    }
                    finish<16>(p.e, bias, v, r, n0, lane, tok0 + c, n - c);
                }
                if (n <= 0) release(b);
                ++j;
            }
        }
    }
    tc_before();
    __syncwarp();
    cluster_sync();                                      // both CTAs' roles have left their loops
    if (cta == 0 && tid == 0) {
        // after a timeout copies may still be in flight: complete the phases of the steps that one of the CTAs has not
        // arrived for and wait, within the limit, for the bytes
        int other_abort, other_issued;
        asm volatile("ld.volatile.shared::cluster.u32 %0, [%1];" : "=r"(other_abort) : "r"(in_peer(su32(&abort_word))) : "memory");
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other_issued) : "r"(in_peer(su32(&issued))) : "memory");
        if (*abort_flag || other_abort) {
            const int last = max(issued, other_issued);
            for (int s = max(0, last - kStages); s < last; ++s) {
                if (issued <= s) mbar_arrive(&full[s % kStages]);
                if (other_issued <= s) mbar_arrive(&full[s % kStages]);
            }
            for (int s = max(0, last - kStages); s < last; ++s) drain_wait(&full[s % kStages], (s / kStages) & 1, p.wait_ns);
            if (p.status) atomicCAS(p.status, (int)MOE_OK, (int)MOE_ERR_TIMEOUT);
        }
    }
    __syncwarp();
    cluster_sync();
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kPairTmem) : "memory");
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

cudaError_t launch_clusters(const void* fn, dim3 grid, int cluster, size_t smem, cudaStream_t s, void** args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

bool fill(LinearParams& p, const LinearArgs& a) {
    const cuuint64_t wd[3] = {(cuuint64_t)(a.in_out ? a.N : a.K), (cuuint64_t)(a.in_out ? a.K : a.N), 1};
    const cuuint64_t ws[2] = {(cuuint64_t)a.w_stride * 2, 0};
    const cuuint64_t xd[3] = {(cuuint64_t)a.K, (cuuint64_t)a.T, 1};
    const cuuint64_t xs[2] = {(cuuint64_t)a.x_stride * 2, 0};
    const CUtensorMapDataType type = a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!encode_map(&p.tw, type, 2, a.w, wd, ws, 64, a.in_out ? 64 : 128)) return false;
    if (!encode_map(&p.tx, type, 2, a.x, xd, xs, 64, 16 << p.box)) return false;
    p.e = Epilogue{a.bias, a.r, a.y, a.bias_type, a.r_type, a.y_type, a.act, a.r_stride, a.y_stride, a.scale, a.res_scale, a.T, a.N};
    p.nk = ceil_div(a.K, kStepK);
    p.bf16 = a.bf16;
    p.status = a.status;
    const WaitCfg wc = wait_cfg();
    p.wait_ns = wc.limit_ns;
    p.stall = wc.stall;
    return true;
}
// Runs of even length, none longer than the output's type allows.
int run_of(int steps, int y_type) {
    const int longest = y_type == MOE_F32 ? kRun32 : kRun16;
    return (ceil_div(steps, ceil_div(steps, longest)) + kPer - 1) / kPer * kPer;     // (whole stages)
}
static_assert(kRun32 % kPer == 0 && kRun16 % kPer == 0, "runs of whole stages");

constexpr int kSplitSmem = 227 * 1024 - 1024;            // dynamic shared memory of split_kernel, at most

// What the choice knows of a GPU is kept for each of the first kDevices of them (others are asked every time): how many clusters
// fit at a time depends on the GPU's own groups of SMs.
constexpr int kDevices = 64;
struct Gpu {
    int device;                                          // -1: none (moe_linear_path answers for a GB300)
    int sms;
};
Gpu current_gpu() {
    static std::atomic<int> known[kDevices];
    Gpu g{-1, 152};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return g;
    }
    if (dev < kDevices) n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return g;
        }
        if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
    }
    return Gpu{dev, n};
}
// Clusters of c CTAs of the split kernel, one an SM, that run at one time.  A cluster lies within one of the GPU's groups
// of SMs, which are not multiples of it: of 8 CTAs 15 fit 152 SMs, of 6 23, of 4 36.  (One more than fit takes twice the time.)
int clusters_at_once(const Gpu& gpu, const void* fn, int c) {
    static std::atomic<int> known[kDevices][9];          // (the same for every form of the kernel: its shared memory decides)
    static const int gb300[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    if (gpu.device < 0) return gb300[c];
    const bool kept = gpu.device < kDevices;
    int n = kept ? known[gpu.device][c].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n - 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c * 64);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return gb300[c];
    }
    if (kept) known[gpu.device][c].store(n + 1, std::memory_order_relaxed);
    return n;
}

// How a product is cut: columns of a tile, and CTAs that share its sum (split) or 0 for the kernel of pairs.
struct Shape {
    int cols, splits;
};
// The least time by a model of both kernels, in us, fitted to graphs of calls on weights that come from HBM (512..7168 wide,
// T = 16..1024; it is within 15 % there).  Outside it is a guide, no more: where x is what streams from memory a step takes longer than
// its constants say (6225 x 4920 -> 328 in tiles of 192: 23 us by the model, 37 measured; of 128 30 and 50):
//   split, of `cols` columns:  start[cols] + (waves - 1) wave[cols] + waves * steps of the sum a CTA * step[cols]
//                              + 0.3 + 0.2 CTAs where they share a sum
//   pairs, of `cols` columns:  3.4 + 0.009 cols + s + (waves - 1) max(s, 0.6 + 0.0063 cols),  s = steps * pair_step(cols)
// The start holds launch, first load and epilogue; what a further wave costs besides its steps is the set-up and epilogue of a CTA
// (pairs: an epilogue longer than the steps that it overlaps; 5521 x 32 -> 3320 in tiles of 32, 64, 128 and 256: 25.3, 17.0, 14.2 and
// 12.3 us; 1000 x 64 -> 1000: split by 16 in 4 waves 8.4, pairs of 64 in one 4.2).  Measured, split / pairs at their best: 16 rows, 2048 -> 2048: 5.6 / 8.4;
// 64 rows, 2048 -> 2048: 6.7 / 8.4, 7168 -> 2048: 10.3 / 20.8; 128 rows, 768 -> 2048: 5.7 / 5.5; 256 rows, 2048 -> 2048: 9.1 / 8.6,
// 768 -> 2048: 6.5 / 5.8, 7168 -> 2048: 16.2 / 20.2, 2048 -> 7168: 22.7 / 12.0; 512 rows, 2048 -> 2048: 11.3 / 9.2.
// (The split kernel with tiles of 128 columns was slower than one or the other at each of these.)
Shape shape_of(const LinearArgs& a, const void* const (&fns)[3]) {
    static const float start[3] = {3.35f, 3.95f, 5.2f}, step[3] = {0.155f, 0.162f, 0.168f}, wave[3] = {2.0f, 2.3f, 5.0f};
    const Gpu gpu = current_gpu();
    const int nk = ceil_div(a.K, kStepK), sms = gpu.sms;
    Shape best{0, 0};
    float least = 1e30f;
    auto take = [&](float t, int cols, int splits) {
        if (t < least) {
            least = t;
            best = Shape{cols, splits};
        }
    };
    for (int i = 0; i < 3 && (16 << i) < 2 * (int64_t)a.T + 16; ++i) {
        const int64_t tiles = (int64_t)ceil_div(a.N, 128) * ceil_div(a.T, 16 << i);
        if (tiles > 4 * sms) continue;
        const int waves = ceil_div(tiles, sms);
        take(start[i] + (waves - 1) * wave[i] + waves * nk * step[i], 16 << i, 1);
        for (int c = 2; c <= 8 && c <= nk && tiles * c <= sms; ++c)
            if (tiles <= clusters_at_once(gpu, fns[i], c)) take(start[i] + 0.3f + 0.2f * c + ceil_div(nk, c) * step[i], 16 << i, c);
    }
    // (beyond some waves, all of them full: the largest tiles)
    for (int nb = ceil_div(a.T, kPairCols), most = std::min(ceil_div(a.T, 32), nb + 64); nb <= most; ++nb) {
        const int cols = (ceil_div(a.T, nb) + 31) & ~31;
        const float per = cols <= 128 ? 0.150f + 0.00014f * cols : 0.117f + 0.00057f * cols;
        const int64_t waves = ceil_div((int64_t)ceil_div(a.N, 256) * ceil_div(a.T, cols), sms / 2);
        take(3.4f + 0.009f * cols + nk * per + (waves - 1) * std::max(nk * per, 0.6f + 0.0063f * cols), cols, 0);
    }
    return best;
}
const void* const kSplit[2][3] = {
    {(const void*)split_kernel<false, 16>, (const void*)split_kernel<false, 32>, (const void*)split_kernel<false, 64>},
    {(const void*)split_kernel<true, 16>, (const void*)split_kernel<true, 32>, (const void*)split_kernel<true, 64>}};

cudaError_t launch_split(const LinearArgs& a, Shape shape, cudaStream_t s) {
    LinearParams p{};
    p.cols = shape.cols;
    p.box = p.cols > 32 ? 2 : p.cols > 16 ? 1 : 0;
    if (!fill(p, a)) return cudaErrorInvalidValue;
    p.n_mb = ceil_div(a.N, 128);
    p.n_tb = ceil_div(a.T, p.cols);
    const void* fn = kSplit[a.in_out][p.box];
    static std::atomic<uint64_t> ready[6];
    int sms = 0;
    cudaError_t err = prepare_kernel(fn, kSplitSmem, ready[3 * a.in_out + p.box], &sms);
    if (err != cudaSuccess) return err;
    const int steps = ceil_div(p.nk, shape.splits), stage = kPer * (kABytes + p.cols * 128), sent = p.cols * 512;
    const int parts = shape.splits > 1 ? ceil_div(p.cols, shape.splits) * shape.splits * 512 : 0;
    p.run = run_of(steps, a.y_type);
    auto fours = [](const void* q, int type, int64_t stride) {
        return !q || ((uintptr_t)q % (type == MOE_F32 ? 16 : 8) == 0 && stride % 4 == 0);
    };
    p.vec = a.N % 4 == 0 && fours(a.y, a.y_type, a.y_stride) && fours(a.r, a.r_type, a.r_stride);
    p.stages = std::min(std::min(ceil_div(steps, kPer), kMaxStages), (kSplitSmem - 1024 - parts) / stage);
    void* args[] = {&p};
    return launch_clusters(fn, dim3(p.n_mb * shape.splits, p.n_tb), shape.splits, 1024 + (size_t)std::max(p.stages * stage, sent) + parts,
                           s, args);
}

cudaError_t launch_pairs(const LinearArgs& a, Shape shape, cudaStream_t s) {
    LinearParams p{};
    static std::atomic<uint64_t> ready[8];
    int sms = 0;
    const bool runs = ceil_div(a.K, kStepK) > (a.y_type == MOE_F32 ? kRun32 : kRun16), wide = shape.cols > 128;
    const int v = (a.in_out ? 4 : 0) + (runs ? 2 : 0) + (wide ? 1 : 0);
    static const void* const fns[8] = {(const void*)pair_kernel<false, false, false>, (const void*)pair_kernel<false, false, true>,
                                       (const void*)pair_kernel<false, true, false>,  (const void*)pair_kernel<false, true, true>,
                                       (const void*)pair_kernel<true, false, false>,  (const void*)pair_kernel<true, false, true>,
                                       (const void*)pair_kernel<true, true, false>,   (const void*)pair_kernel<true, true, true>};
    const void* fn = fns[v];
    const int smem = 1024 + (wide ? kPairStages<true> * kPairPer<true> * kPairStep<true> : kPairStages<false> * kPairPer<false> * kPairStep<false>);
    cudaError_t err = prepare_kernel(fn, smem, ready[v], &sms);
    if (err != cudaSuccess) return err;
    p.cols = shape.cols;
    p.box = p.cols > 128 ? 3 : p.cols > 64 ? 2 : p.cols > 32 ? 1 : 0;
    if (!fill(p, a)) return cudaErrorInvalidValue;
    p.n_mb = ceil_div(a.N, 256);
    p.n_tb = ceil_div(a.T, p.cols);
    p.run = run_of(p.nk, a.y_type);
    const int64_t tiles = (int64_t)p.n_mb * p.n_tb;
    void* args[] = {&p};
    return launch_early(fn, dim3(2 * (unsigned)std::min<int64_t>(tiles, sms / 2)), runs ? kPairThreads<true> : kPairThreads<false>, smem,
                        s, args);
}

}  // namespace

bool linear_pairs(const LinearArgs& a) { return shape_of(a, kSplit[a.in_out]).splits == 0; }

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    const Shape shape = shape_of(a, kSplit[a.in_out]);
    return shape.splits ? launch_split(a, shape, s) : launch_pairs(a, shape, s);
}

}  // namespace moe
