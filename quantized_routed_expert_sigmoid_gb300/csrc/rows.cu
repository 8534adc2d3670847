// rows.cu -- products of a few rows per expert with bf16 / fp16 weights: the weights of the
// experts that have rows are streamed once through registers.
//
//   y[i, n] = sum_c W[e][n, c] v_i[c],  or  silu(W v) * (W_up v),   v_i = x[sorted_pairs[i] / k] or x[i]
//
// Bound: the weights' bytes.  A decode step multiplies each weight with one to a few rows, so the
// only question is how fast HBM can be kept busy; the arithmetic rides on the warps' matrix
// instruction m16n8k16 (weights as the 16-row operand, up to 8 rows of x as its columns), whose
// operands are registers: a weight goes from its 16-byte load to the instruction without a stop in
// shared memory.  (tcgen05 would need it staged there, which costs more than it saves here.)
// The sum over c may run in any order, so the operands' k slots are filled in the order in which the
// weights lie in memory: lane (g, t) of a warp holds 16 consecutive bytes of weight row g, and the
// same elements of x row g, and no element is moved between lanes.
// Layout: a CTA of 8 warps takes 32 weight rows (16 of W and the same 16 of W_up when gated; 64
// for [in][out] weights, which come here ungated) of one expert; the warps split the sum over c and join in shared
// memory at the end, in a fixed order.
// Measured: one token, 8 of 128 experts, 2048 -> 768 gated, bf16: 11.8 us for 50 MB (7.5 us at the copy's
// rate); three CTAs an SM with two chunks in flight a warp, so that all 384 run at once (with one to two CTAs and four
// chunks: 16.0 us).  What is left is the start: the offsets, the pair and the first weights follow one another.
#include "products.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Streamed weights: read once, not kept in L1.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Elements i .. i + 7 of a 16-bit row of n elements (zeros past its end): 16 bytes at a time, single
// elements where the row ends inside the eight.
template <bool STREAM>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int i, int n) {
    if (i + 8 <= n) return STREAM ? ld_stream16(row + i) : __ldg(reinterpret_cast<const uint4*>(row + i));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) w[j >> 1] |= (uint32_t)__ldg(row + i + j) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Elements i .. i + 3 (i a multiple of 4; rows start on 16 bytes).
__device__ __forceinline__ uint2 load4(const uint16_t* row, int i, int n) {
    if (i + 4 <= n) return __ldg(reinterpret_cast<const uint2*>(row + i));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + j < n) w[j >> 1] |= (uint32_t)__ldg(row + i + j) << (16 * (j & 1));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void raise(int32_t* status) {
    if (status) atomicCAS(status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
}

// The slot-th expert that has rows: its id and range of sorted positions (n = 0: there is none).
// Offsets are clamped into 0..P.  All threads of the CTA call it.
__device__ __forceinline__ void find_expert(const RowsArgs& a, int slot, int& e_out, int& lo_out, int& n_out) {
    __shared__ int s_cnt[kWarps], s_e, s_lo, s_n;
    if (!a.offsets) { e_out = 0; lo_out = 0; n_out = slot == 0 ? a.P : 0; return; }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_n = 0;
    int seen = 0;
    bool bad = false;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + tid;
        int lo = 0, n = 0;
        if (e < a.E) {
            const int o0 = __ldg(a.offsets + e), o1 = __ldg(a.offsets + e + 1);
            bad |= o0 < 0 || o1 < o0 || o1 > a.P;
            lo = min(max(o0, 0), a.P);
            n = max(min(max(o1, 0), a.P) - lo, 0);
        }
        const unsigned m = __ballot_sync(0xffffffffu, n > 0);
        __syncthreads();                               // (s_cnt of the round before has been read)
        if (lane == 0) s_cnt[warp] = __popc(m);
        __syncthreads();
        int base = seen;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += s_cnt[w];
            seen += s_cnt[w];
        }
        if (n > 0 && base + __popc(m & ((1u << lane) - 1u)) == slot) { s_e = e; s_lo = lo; s_n = n; }
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) raise(a.status);
    __syncthreads();
    e_out = s_e; lo_out = s_lo; n_out = s_n;
}

// Row of x for sorted position i.
__device__ __forceinline__ int64_t x_row(const RowsArgs& a, int i) {
    if (!a.sorted_pairs) return i;
    const int p = __ldg(a.sorted_pairs + i);
    if (p < 0 || p >= a.P) { raise(a.status); return 0; }
    return p / a.k;
}

// ------------------------------------------------------------------ the sum over c
// Each fills acc[mat][tile][nt] (m16n8 accumulators: c0, c1 = row g, columns 2t, 2t + 1; c2, c3 = row
// g + 8) with this warp's share.  xr[j]: this lane's row of x in column tile j (NULL: none).

// The matrix instruction cuts its sum off instead of rounding it, an error towards zero that grows with the number of
// instructions in a row (8.6e-7, gated 1.7e-6, at 7168 elements); so what a warp loads at once is summed by
// itself and added with rounding.
template <int TI, int NT>
__device__ __forceinline__ void add(float (&acc)[TI][NT][4], const float (&part)[TI][NT][4]) {
#pragma unroll
    for (int j = 0; j < TI; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][n][i] += part[j][n][i];
}

// [out][in] weights: warps take chunks of 32 c, lane (g, t) 8 of them of rows g and g + 8.
template <bool BF16, bool UP, int NT>
struct OutIn {
    static constexpr int kMats = UP ? 2 : 1, kTiles = UP ? 1 : 2, kRows = 16 * kTiles, kCtas = 3;
    __device__ static __forceinline__ int row(int tile, int g, int half) { return 16 * tile + g + 8 * half; }
    __device__ static __forceinline__ void run(const RowsArgs& a, int e, int r0, const uint16_t* const (&xr)[NT],
                                               int nt, float (&acc)[kMats][kTiles][NT][4]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        const uint16_t* wr[2][2];                       // [mat or tile][half]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = min(r0 + row(UP ? 0 : j, g, h), a.N - 1);      // (rows past the end are not stored)
                wr[j][h] = static_cast<const uint16_t*>(UP && j == 1 ? a.w1 : a.w0) + (int64_t)e * a.expert_stride +
                           (int64_t)r * a.row_stride;
            }
        constexpr int U = NT == 1 ? 2 : 4;              // chunks in flight
        const int n_chunks = (a.K + 31) / 32;
        for (int c0 = warp; c0 < n_chunks; c0 += U * kWarps) {
            uint4 w[U][2][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (c0 + u * kWarps) * 32 + 8 * t;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[u][j][h] = load8<true>(wr[j][h], i, a.K);
            }
            float part[kMats][kTiles][NT][4] = {};      // (see add)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (c0 + u * kWarps) * 32 + 8 * t;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n >= nt) break;
                    const uint4 b = xr[n] ? load8<false>(xr[n], i, a.K) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float(&c)[4] = part[UP ? j : 0][UP ? 0 : j][n];
                        mma16816<BF16>(c, w[u][j][0].x, w[u][j][1].x, w[u][j][0].y, w[u][j][1].y, b.x, b.y);
                        mma16816<BF16>(c, w[u][j][0].z, w[u][j][1].z, w[u][j][0].w, w[u][j][1].w, b.z, b.w);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < kMats; ++m) add(acc[m], part[m]);
        }
    }
};

// [in][out] weights (one matrix: the gated pair is the tensor-core kernel's): warps take chunks of 16 c; lane (g, t)
// holds outputs 8g .. 8g + 7 of c = 4t .. 4t + 3, and byte permutes pair the c of one output.  Output 8g + 2 tile + half
// is row g + 8 half.
template <bool BF16, int NT>
struct InOut {
    static constexpr int kMats = 1, kTiles = 4, kRows = 64, kCtas = 2;
    __device__ static __forceinline__ int row(int tile, int g, int half) { return 8 * g + 2 * tile + half; }
    __device__ static __forceinline__ void run(const RowsArgs& a, int e, int r0, const uint16_t* const (&xr)[NT],
                                               int nt, float (&acc)[kMats][kTiles][NT][4]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        constexpr int U = 4;
        const int n_chunks = (a.K + 15) / 16, n0 = r0 + 8 * g;
        const uint16_t* p = static_cast<const uint16_t*>(a.w0) + (int64_t)e * a.expert_stride;
        for (int c0 = warp; c0 < n_chunks; c0 += U * kWarps) {
            uint4 w[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (c0 + u * kWarps) * 16 + 4 * t;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    w[u][r] = i + r < a.K ? load8<true>(p + (int64_t)(i + r) * a.row_stride, n0, a.N) : make_uint4(0u, 0u, 0u, 0u);
            }
            float part[kTiles][NT][4] = {};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (c0 + u * kWarps) * 16 + 4 * t;
                const uint32_t* q0 = &w[u][0].x;
                const uint32_t* q1 = &w[u][1].x;
                const uint32_t* q2 = &w[u][2].x;
                const uint32_t* q3 = &w[u][3].x;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n >= nt) break;
                    const uint2 b = xr[n] ? load4(xr[n], i, a.K) : make_uint2(0u, 0u);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma16816<BF16>(part[j][n], __byte_perm(q0[j], q1[j], 0x5410), __byte_perm(q0[j], q1[j], 0x7632),
                                       __byte_perm(q2[j], q3[j], 0x5410), __byte_perm(q2[j], q3[j], 0x7632), b.x, b.y);
                }
            }
            add(acc[0], part);
        }
    }
};

template <class W, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? W::kCtas : 1) rows_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int kMats = W::kMats, kTiles = W::kTiles, kFrag = kTiles * 4;
    __shared__ float red[kWarps][kMats * kFrag][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2;
    int e, lo, cnt;
    wait_for_previous();
    allow_next();
    find_expert(a, blockIdx.y, e, lo, cnt);
    if (cnt == 0) return;
    const int r0 = blockIdx.x * W::kRows;
    for (int base = 0; base < cnt; base += 8 * NT) {
        const int nt = min(NT, (cnt - base + 7) / 8);
        const uint16_t* xr[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int i = base + 8 * n + g;
            xr[n] = i < cnt ? static_cast<const uint16_t*>(a.x) + x_row(a, lo + i) * a.x_stride : nullptr;
        }
        float acc[kMats][kTiles][NT][4];
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][j][n][i] = 0.f;
        W::run(a, e, r0, xr, nt, acc);
        // join the warps' shares, in the warps' order, one column tile at a time
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt) break;
            __syncthreads();
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) red[warp][m * kFrag + 4 * j + i][lane] = acc[m][j][n][i];
            __syncthreads();
            for (int f = warp; f < kFrag; f += kWarps) {
                float v[kMats];
#pragma unroll
                for (int m = 0; m < kMats; ++m) {
                    v[m] = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v[m] += red[w][m * kFrag + f][lane];
                }
                const int col = base + 8 * n + 2 * (lane & 3) + (f & 1), r = r0 + W::row(f >> 2, g, (f >> 1) & 1);
                if (col < cnt && r < a.N) {
                    float out = v[0];
                    if constexpr (kMats == 2) out = silu_times<false>(v[0], v[1]);
                    store_value(a.y, a.y_type, (int64_t)(lo + col) * a.y_stride + r, out);
                }
            }
        }
    }
}

template <class W, int NT>
cudaError_t launch(const RowsArgs& a, cudaStream_t s) {
    const dim3 grid((a.N + W::kRows - 1) / W::kRows, a.offsets ? min(a.E, a.P) : 1);
    void* args[] = {const_cast<RowsArgs*>(&a)};
    return launch_early((const void*)rows_kernel<W, NT>, grid, kThreads, 0, s, args);
}
template <bool BF16, bool UP>
cudaError_t launch_w(const RowsArgs& a, cudaStream_t s) {
    // columns held at once: what an expert can have at most (a token asks for an expert once, so T rows;
    // more than the columns are taken in passes).  [in][out] weights come here ungated, with less than 8 rows in all.
    const int most = a.offsets ? a.P / a.k : a.P;
    if constexpr (!UP)
        if (a.in_out) return launch<InOut<BF16, 1>, 1>(a, s);
    if (most <= 8) return launch<OutIn<BF16, UP, 1>, 1>(a, s);
    return launch<OutIn<BF16, UP, 2>, 2>(a, s);
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
    if (a.P <= 0) return cudaSuccess;
    if (a.bf16) return a.w1 ? launch_w<true, true>(a, s) : launch_w<true, false>(a, s);
    return a.w1 ? launch_w<false, true>(a, s) : launch_w<false, false>(a, s);
}

}  // namespace moe
