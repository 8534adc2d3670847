// w4.cu -- products of a few rows per expert with 4-bit weights and group scales.
//
//   y[i, n] = sum_g s[n, g] * sum_{c in g} (q[n, c] - z[n, g]) v_i[c]
// (and silu(W v) * (W_up v) of two such products), v_i = x[sorted_pairs[i] / k] or x[i].
//
// Bound: the bytes of the codes and scales; next to that the instructions that turn a code into an
// operand.  Both shape the kernel:
// - Codes come by TMA into a ring of shared memory (128 rows x 256 codes a stage, six stages in flight
//   a SM), so that the reads in flight do not depend on registers.  128-byte swizzled rows make the
//   warps' reads of 8 rows x 16 bytes free of bank conflicts.
// - The products run on the warps' m16n8k16 instruction, weights as the 16-row operand (8 rows of W
//   and the same 8 of W_up when gated, so that both halves of an output meet in one thread), up to 8 rows of
//   x as its columns.  Its sum over c may run in any order, so codes are used in the order in which they lie: nibbles
//   j and j + 4 of a 32-bit word become the 16-bit halves of an operand register.  Put into the low bits of 1024.0 in
//   fp16 a nibble is 1024 + q (or, four bits higher, 1024 + 16 q); adding -1024 - z (or multiplying by 1/16 and
//   adding -64 - z) leaves q - z, exactly: one mask, one packed addition and half a shift an operand.
// - So a weight that equals its zero point is a 0 and adds nothing, whatever x is there.  (Taking z sum x off sum q x
//   instead, with the codes as they are, saved the addition, but both sums are rounded to their own size: a
//   channel of x far above the others whose codes equal the zero point left an error in proportion to it,
//   8.6e-4 of the result at 20000 times the others.)
// - A group's sum is at most two chains of four instructions, and the scale is applied to it in fp32.
// - x is staged once per expert as fp16, in the word order of the codes: bf16 rows scaled by a power of two so that their
//   largest finite magnitude is 2^14 to 2^15 (a value keeps all its bits down to 2^-31 of the largest), fp16 rows
//   scaled up only, which loses nothing.
// 8 computing warps (4 sets of 32 weight rows, every other stage each, joined at the end of a unit), one warp
// that issues the codes' copies and three that copy scales and zero points, a stage each in turn (one warp for
// both took 1400 clocks a stage); a CTA per SM takes an even share of the (expert, 128 rows) units.
//
// Measured (device time): 16 tokens, 8 of 256 experts, 7168 -> 2048 gated, groups of 32 with zero points:
// 438 us for 1.78 GB (266 us at the copy's rate; 385 us with the zero points taken off the sums).  What bounds it now is the issue of
// instructions: two computing warps a scheduler find one to issue in 61 % of the clocks (32 experts of that size, one row each: DRAM 48 %,
// ALU pipe 58 %), and every instruction more shows (8 additions a group: 478 us); the 128 matrix instructions of
// a stage, one in 16 clocks on each of the four schedulers, take 512 of the 700 clocks that HBM needs for it beside that.
// One token, 8 of 128 experts, 2048 -> 768 gated, groups of 128: 9.2 us for 13 MB; 96 units of 64 outputs leave 56 of
// 152 SMs without work, and each CTA's eight stages follow a start of 4 us (routing read, x staged, the first copies).
#include <type_traits>

#include "products.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kRowWarps = 4, kWarps = 2 * kRowWarps;     // computing warps: sets of rows x alternate stages
constexpr int kTiles = 2, kScaleWarps = 3, kAllWarps = kWarps + 1 + kScaleWarps, kThreads = 32 * kAllWarps;
constexpr int kStages = 6, kStageBytes = 128 * 128, kStageK = 256;
constexpr int kSmemMax = 227 * 1024;

// A word's nibbles 0 and 4 (1 and 5) as the halves of q - z: nz is -1024 - z (-64 - z) in both halves.
__device__ __forceinline__ uint32_t low_codes(uint32_t v, uint32_t nz) {
    const uint32_t m = (v & 0x000F000Fu) | 0x64006400u;      // 1024 + q
    const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&nz));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t v, uint32_t nz) {
    const uint32_t m = (v & 0x00F000F0u) | 0x64006400u, sixteenth = 0x2C002C00u;   // 1024 + 16 q
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&sixteenth),
                              *reinterpret_cast<const __half2*>(&nz));
    return *reinterpret_cast<const uint32_t*>(&r);
}
struct W4Params {
    CUtensorMap tw0, tw1;        // codes of W and W_up: [E * N][K / 2] bytes, boxes of 128 bytes x 128 (gated: 64) rows
    RowsArgs a;
    int cols;                    // rows of x staged at once
    int x_stride;                // bytes between staged rows
    bool vec;                    // scales and zero points can be read a stage's share at a time
    uint64_t wait_ns;
    int stall;
};

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zero.
__device__ __forceinline__ void mma_f16_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Reads of shared memory by 32-bit address.
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
// 16 bytes where `on` holds, else v stays as it was.
__device__ __forceinline__ void lds16_if(uint4& v, uint32_t a, bool on) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n @p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n}\n"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "r"(a), "r"((uint32_t)on));
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void computing_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// Bytes of a row's scales and zero points in a stage (a copy has at least 4 bytes: with groups of 128 the two
// zero points are copied with the two before or after them).
template <int G>
__host__ __device__ constexpr int scale_bytes() { return kStageK / G * 2; }
template <int G>
__host__ __device__ constexpr int zero_bytes() { return G == 128 ? 4 : kStageK / G; }
template <int G>
__host__ __device__ constexpr int stage_scales() { return 128 * (scale_bytes<G>() + zero_bytes<G>()); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// BYTES of shared memory as words.
template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t* v) {
    if constexpr (BYTES == 16) {
        const uint4 w = lds16(a);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else if constexpr (BYTES == 8) {
        const uint2 w = lds8(a);
        v[0] = w.x; v[1] = w.y;
    } else {
        v[0] = lds4(a);
    }
}

template <int G, bool UP, int NT, bool SCALE_BF16>
__global__ void __launch_bounds__(kThreads, 1) w4_kernel(const __grid_constant__ W4Params p) {
    constexpr int kCols = 8 * NT, kUnit = UP ? 64 : 128;   // outputs of a unit
    constexpr int kGroups = kStageK / G;                   // groups of a stage
    constexpr int kJoin = kTiles * 4 * NT * 32 * kRowWarps;
    const RowsArgs& a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int n_groups = a.K / G, n_ks = (a.K + kStageK - 1) / kStageK;
    uint8_t* scales = ring_base + kStages * kStageBytes;   // [stages] scales, then zero points, of 128 rows
    uint8_t* xs = scales + kStages * stage_scales<G>();    // staged x: p.cols rows, p.x_stride bytes apart
    float* unscale = reinterpret_cast<float*>(xs + (size_t)p.cols * p.x_stride);   // [kCols] the rows' powers of two
    float* join = unscale + kCols;                         // [2][kTiles * 4 * NT][32 * kRowWarps] one of two warps' sums
    float* largest = join + 2 * kJoin;                     // [kWarps]
    uint64_t* full = reinterpret_cast<uint64_t*>(largest + kWarps);
    uint64_t* empty = full + kStages;
    uint64_t* never = empty + kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
    int* cnt = reinterpret_cast<int*>(never + 2);          // [kAllWarps]
    int* done = cnt + kAllWarps;                           // [kScaleWarps] last step + 1 that a scale warp has arrived for
    int* off = cnt + 20;                                   // [E + 1]
    uint16_t* expert = reinterpret_cast<uint16_t*>(off + a.E + 1);   // [E] those with rows

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1 + 32); mbar_init(&empty[i], kRowWarps); }
        mbar_init(never, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous();
    allow_next();
    // ---- the experts that have rows
    bool bad = false;
    for (int i = tid; i <= a.E; i += kThreads) {
        const int o = a.offsets ? __ldg(a.offsets + i) : (i ? a.P : 0);
        bad |= o < 0 || o > a.P || (i > 0 && a.offsets && __ldg(a.offsets + i - 1) > o);
        off[i] = min(max(o, 0), a.P);
    }
    __syncthreads();
    int n_active = 0;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + tid;
        const bool has = e < a.E && off[e + 1] > off[e];
        const unsigned m = __ballot_sync(0xffffffffu, has);
        if (lane == 0) cnt[warp] = __popc(m);
        __syncthreads();
        int inc = lane < kAllWarps ? cnt[lane] : 0;
        const int own = inc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const int base = n_active + __shfl_sync(0xffffffffu, inc - own, warp);
        n_active += __shfl_sync(0xffffffffu, inc, 31);
        if (has) expert[base + __popc(m & ((1u << lane) - 1u))] = (uint16_t)e;
        __syncthreads();
    }
    // this CTA's units: an even share (at most 2^10 experts x 2^14 blocks in all)
    const uint32_t n_blk = (uint32_t)(a.N + kUnit - 1) / kUnit, units = n_active * n_blk;
    const uint32_t share = units / gridDim.x, more = units - share * gridDim.x;
    const uint32_t u0 = share * blockIdx.x + min(blockIdx.x, more), u1 = u0 + share + (blockIdx.x < more ? 1 : 0);

    // Bounded wait; after a wait has run out every wait returns at once and the loops run to their ends, so that the
    // CTA's barriers stay matched: nothing more is copied into the ring, no warp arrives for a step that it has not
    // filled, and nothing is stored.
    auto wait = [&](uint64_t* b, uint32_t parity) {
        for (int i = 0; i < 64; ++i) {
            if (mbar_test(b, parity)) return;
            if (*abort_flag) return;
        }
        const uint64_t t0 = gtime();
        while (!mbar_test(b, parity)) {
            if (*abort_flag) return;
            if (gtime() - t0 > p.wait_ns) { *abort_flag = 1; return; }
        }
    };
    int s = 0, n_issued = 0, step = 0, last = 0;
    uint32_t ph = 0;
    for (uint32_t u = u0; u < u1;) {
        // the units of one expert
        const int nth = u / n_blk, e = expert[nth], b0 = (int)(u - nth * n_blk);
        const int b1 = (int)min(n_blk, b0 + (u1 - u));
        const int lo = off[e], rows = off[e + 1] - lo;
        u += b1 - b0;
        for (int base = 0; base < rows; base += p.cols) {
            if (warp == kWarps) {
                // ======================= codes =======================
                for (int b = b0; b < b1; ++b)
                    for (int ks = 0; ks < n_ks; ++ks) {
                        wait(&empty[s], ph ^ 1);
                        __syncwarp();
                        if (!__any_sync(0xffffffffu, *abort_flag)) {
                            if (lane == 0) {
                                mbar_expect_tx(&full[s], kStageBytes);
                                uint8_t* dst = ring_base + s * kStageBytes;
                                const int row = e * a.N + b * kUnit;
                                tma_load_2d(dst, &p.tw0, ks * 128, row, &full[s]);
                                if constexpr (UP) tma_load_2d(dst + 8192, &p.tw1, ks * 128, row, &full[s]);
                                mbar_arrive(&full[s]);
                            }
                            ++n_issued;
                        }
                        if (++s == kStages) { s = 0; ph ^= 1; }
                    }
                continue;
            }
            if (warp > kWarps) {
                // ======================= scales and zero points =======================
                for (int b = b0; b < b1; ++b) {
                    // lane u brings the scales of rows u, u + 32, ..
                    int64_t at[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = ((int64_t)e * a.N + min(b * kUnit + (UP ? (32 * i + lane) & 63 : 32 * i + lane), a.N - 1)) * n_groups;
                    for (int ks = 0; ks < n_ks; ++ks) {
                        bool mine = step % kScaleWarps == warp - kWarps - 1;
                        ++step;
                        if (mine) {
                            wait(&empty[s], ph ^ 1);
                            __syncwarp();
                            mine = !__any_sync(0xffffffffu, *abort_flag);
                        }
                        if (mine) {
                            last = step;
                            uint8_t* to = scales + s * stage_scales<G>();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint16_t* sp = static_cast<const uint16_t*>(UP && i >= 2 ? a.s1 : a.s0) + at[i] + ks * kGroups;
                                const uint8_t* zp = (UP && i >= 2 ? a.z1 : a.z0) + at[i] + ks * kGroups;
                                uint8_t* ts = to + (32 * i + lane) * scale_bytes<G>();
                                uint8_t* tz = to + 128 * scale_bytes<G>() + (32 * i + lane) * zero_bytes<G>();
                                if (p.vec) {
                                    copy_async<scale_bytes<G>()>(su32(ts), sp);
                                    if (a.z0) {
                                        if constexpr (G == 128) copy_async<4>(su32(tz), reinterpret_cast<const void*>((uintptr_t)zp & ~(uintptr_t)3));
                                        else copy_async<zero_bytes<G>()>(su32(tz), zp);
                                    }
                                } else {
#pragma unroll
                                    for (int q = 0; q < kGroups; ++q) {
                                        const bool in = ks * kGroups + q < n_groups;
                                        reinterpret_cast<uint16_t*>(ts)[q] = in ? __ldg(sp + q) : (uint16_t)0;
                                        if (a.z0) tz[q] = in ? __ldg(zp + q) : (uint8_t)0;
                                    }
                                }
                            }
                            if (p.vec) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(&full[s])) : "memory");
                            else mbar_arrive(&full[s]);
                        }
                        if (++s == kStages) { s = 0; ph ^= 1; }
                    }
                }
                cp_wait_all();
                continue;
            }
            // ======================= staging of x =======================
            const int nc = min(p.cols, rows - base);
            computing_sync();                            // the rows before have been used
            // a set of wc warps a row: all 8 for one row, one each for 5 and more (more than one: all rows at once)
            int wc = kWarps;
            while (wc > 1 && wc * nc > kWarps) wc >>= 1;
            for (int c0 = 0; c0 < nc; c0 += kWarps / wc) {
                const int c = c0 + warp / wc, sub = warp % wc;
                const int step = 256 * wc, i0 = 8 * (32 * sub + lane);
                const uint16_t* src = static_cast<const uint16_t*>(a.x);
                if (c < nc) {
                    int64_t row = lo + base + c;
                    if (a.sorted_pairs) {
                        const int pair = __ldg(a.sorted_pairs + row);
                        const bool in = (uint32_t)pair < (uint32_t)a.P;
                        bad |= !in;
                        row = in ? pair / a.k : 0;
                    }
                    src += row * a.x_stride;
                }
                auto load = [&](int i) {
                    return c < nc && i < a.K ? __ldg(reinterpret_cast<const uint4*>(src + i)) : make_uint4(0u, 0u, 0u, 0u);
                };
                auto values = [&](const uint4& w, float (&v)[8]) {
                    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (a.bf16) {
                            v[2 * j] = __uint_as_float(r[j] << 16);
                            v[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[j]));
                            v[2 * j] = f.x;
                            v[2 * j + 1] = f.y;
                        }
                    }
                };
                constexpr int kHold = 4;                 // reads a thread has in flight (and keeps, if they are all)
                uint4 held[kHold];
                float most = 0.f;
                for (int i = i0; i < a.K; i += kHold * step) {
#pragma unroll
                    for (int h = 0; h < kHold; ++h) held[h] = load(i + h * step);
#pragma unroll
                    for (int h = 0; h < kHold; ++h) {
                        if (i + h * step - 8 * lane >= a.K) break;           // (the same for the whole warp)
                        float v[8];
                        values(held[h], v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[j]) <= 3.402823466e38f ? fabsf(v[j]) : 0.f);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (wc > 1) {
                    if (lane == 0) largest[warp] = most;
                    computing_sync();
                    for (int w = 0; w < wc; ++w) most = fmaxf(most, largest[warp - sub + w]);
                }
                // the largest finite magnitude becomes 2^14 .. 2^15 (that of a tiny row less: its values are exact all the
                // same); infinities and NaN stay what they are
                const int mexp = (int)(__float_as_uint(most) >> 23);
                const int ex = min(max(mexp - 127 - 14, -120), a.bf16 ? 113 : 0);
                const float scale = __int_as_float((127 - ex) << 23);
                if (c < nc && sub == 0 && lane == 0) unscale[c] = __int_as_float((127 + ex) << 23);
                const bool kept = kHold * step >= a.K;
                for (int i = i0; i - 8 * lane < n_ks * kStageK; i += kHold * step) {
                    if (!kept) {
#pragma unroll
                        for (int h = 0; h < kHold; ++h) held[h] = load(i + h * step);
                    } else if (i0 >= a.K) {
#pragma unroll
                        for (int h = 0; h < kHold; ++h) held[h] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int h = 0; h < kHold; ++h) {
                        const int at = i + h * step;
                        if (at - 8 * lane >= n_ks * kStageK) break;          // (the same for the whole warp)
                        float v[8];
                        values(held[h], v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] *= scale;
                        const __half2 h0 = __floats2half2_rn(v[0], v[4]), h1 = __floats2half2_rn(v[1], v[5]);
                        const __half2 h2 = __floats2half2_rn(v[2], v[6]), h3 = __floats2half2_rn(v[3], v[7]);
                        if (c < nc && at < n_ks * kStageK)
                            *reinterpret_cast<uint4*>(xs + (size_t)c * p.x_stride + 2 * at) =
                                make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                                           *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3));
                    }
                }
            }
            computing_sync();
            // ======================= products =======================
            const int rw = warp % kRowWarps, kh = warp / kRowWarps, nt = (nc + 7) / 8;
            const uint32_t xs0 = su32(xs) + t * (G / 2);   // (t * G / 4 elements)
            uint32_t xc[NT];                             // this lane's rows of x (columns without one are not read: their
            bool has[NT];                                // sums are not stored)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                has[n] = 8 * n + g < nc;
                xc[n] = xs0 + (uint32_t)(min(8 * n + g, nc - 1) * p.x_stride);
            }
            // Lane g's row of eight: the lanes whose reads go out together (8 lanes of 16 bytes, 16 of 8, 32 of 4) need
            // rows whose swizzles keep them in different banks: two rows that differ in bit 2, four in bits 1 and 2.
            const int gr = G == 128 ? (g & 1) << 2 | g >> 1 : G == 64 ? (g & 3) << 1 | g >> 2 : g;
            // tile j of this warp: the row of W at ra[j] of the stage, and that of W_up (or the one 8 further)
            int ra[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) ra[j] = (UP ? 8 : 16) * (kTiles * rw + j) + gr;
            // this lane's 16 (8, 4) bytes of a row's group q lie at (this address) xor (q * G / 2): the swizzle
            // exchanges 16-byte chunks by the row's last three bits, which are gr
            const uint32_t ring0 = su32(ring_base) + ra[0] * 128 + (((t * (G / 8)) >> 4 ^ gr) << 4) + ((t * (G / 8)) & 15);
            const uint32_t scales0 = su32(scales) + ra[0] * scale_bytes<G>();
            const uint32_t zeros0 = su32(scales) + 128 * scale_bytes<G>() + ra[0] * zero_bytes<G>();
            constexpr int kTileStep = UP ? 8 : 16, kHalfStep = UP ? 64 : 8;       // rows between tiles and halves
            int turn = 0;
            for (int b = b0; b < b1; ++b, turn ^= 1) {
                float acc[kTiles][NT][4];
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j][n][i] = 0.f;
                for (int ks = 0; ks < n_ks; ++ks) {
                    const bool mine = ((step + kh) & 1) == 0;
                    ++step;
                    if (!mine) {
                        if (++s == kStages) { s = 0; ph ^= 1; }
                        continue;
                    }
                    const bool stalled = p.stall && u - b1 + b == u0 && ks == 0;      // (test setting)
                    wait(stalled ? never : &full[s], stalled ? 0u : ph);
                    const uint32_t codes = ring0 + s * kStageBytes;
                    const uint32_t xk = (uint32_t)(ks * kStageK * 2);
                    // the rows' scales and zero points: [tile][half]
                    constexpr int kS = scale_bytes<G>() / 4, kZ = zero_bytes<G>() / 4;
                    uint32_t fs[kTiles][2][kS], fz[kTiles][2][kZ];
                    const uint32_t so = s * stage_scales<G>();
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            lds_words<scale_bytes<G>()>(scales0 + so + (j * kTileStep + h * kHalfStep) * scale_bytes<G>(), fs[j][h]);
#pragma unroll
                            for (int i = 0; i < kZ; ++i) fz[j][h][i] = 0x08080808u;
                            if (a.z0) {
                                lds_words<zero_bytes<G>()>(zeros0 + so + (j * kTileStep + h * kHalfStep) * zero_bytes<G>(), fz[j][h]);
                                if (G == 128 && p.vec) { // (which half of the four was meant)
                                    const int row = min(b * kUnit + (UP ? ra[j] : ra[j] + 8 * h), a.N - 1);
                                    const uintptr_t at = (uintptr_t)(UP && h ? a.z1 : a.z0) + ((size_t)e * a.N + row) * n_groups;
                                    fz[j][h][0] >>= 8 * ((at + ks * kGroups) & 2);
                                }
#pragma unroll
                                for (int i = 0; i < kZ; ++i) fz[j][h][i] &= 0x0F0F0F0Fu;
                            }
                        }
                    // one group of the stage.  kind: 0 for a single row of x, else column tiles
                    auto group = [&](int q, auto kind) {
                        constexpr int kKind = decltype(kind)::value, NA = kKind == 0 ? 1 : kKind, kWords = G / 32;
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        // this lane's quarter of the group's codes, of every row
                        uint32_t v[kTiles][2][kWords];
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                lds_words<G / 8>((codes ^ (uint32_t)(q * (G / 2))) + (j * kTileStep + h * kHalfStep) * 128, v[j][h]);
                        // -1024 - z and -64 - z of the rows, in both halves
                        uint32_t nz[kTiles][2], nz64[kTiles][2];
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                nz[j][h] = __byte_perm(fz[j][h][q >> 2], 0xE4E4E4E4u, 0x4040u + (q & 3) * 0x0101u);
                                const uint32_t k960 = 0x63806380u;
                                const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&nz[j][h]), *reinterpret_cast<const __half2*>(&k960));
                                nz64[j][h] = *reinterpret_cast<const uint32_t*>(&r);
                            }
                        // (two chains of products, of the low and of the high halves of the words)
                        float part[kTiles][NA][4], high[kTiles][NA][4];
#pragma unroll
                        for (int w = 0; w < kWords; ++w)
#pragma unroll
                            for (int n = 0; n < NA; ++n) {
                                lds16_if(x, xc[n] + xk + 2 * (q * G + 8 * w), has[n]);
#pragma unroll
                                for (int j = 0; j < kTiles; ++j) {
                                    const uint32_t va = v[j][0][w], vb = v[j][1][w];
                                    const uint32_t a0 = low_codes(va, nz[j][0]), a1 = high_codes(va, nz64[j][0]);
                                    const uint32_t a2 = low_codes(va >> 8, nz[j][0]), a3 = high_codes(va >> 8, nz64[j][0]);
                                    const uint32_t b0 = low_codes(vb, nz[j][1]), b1 = high_codes(vb, nz64[j][1]);
                                    const uint32_t b2 = low_codes(vb >> 8, nz[j][1]), b3 = high_codes(vb >> 8, nz64[j][1]);
                                    float(&lo)[4] = part[j][n];
                                    float(&hi)[4] = kWords > 1 ? high[j][n] : part[j][n];
                                    if (w == 0) mma_f16_16816_first(lo, a0, b0, a1, b1, x.x, x.y);
                                    else mma_f16_16816(lo, a0, b0, a1, b1, x.x, x.y);
                                    if (w == 0 && kWords > 1) mma_f16_16816_first(hi, a2, b2, a3, b3, x.z, x.w);
                                    else mma_f16_16816(hi, a2, b2, a3, b3, x.z, x.w);
                                }
                            }
#pragma unroll
                        for (int n = 0; n < NA; ++n)
#pragma unroll
                            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t sw = fs[j][h][q >> 1];
                                    float f;
                                    if constexpr (SCALE_BF16) {
                                        f = __uint_as_float(q & 1 ? sw & 0xFFFF0000u : sw << 16);
                                    } else {
                                        const __half2 hw = *reinterpret_cast<const __half2*>(&sw);
                                        f = q & 1 ? __high2float(hw) : __low2float(hw);
                                    }
                                    float p0 = part[j][n][2 * h], p1 = part[j][n][2 * h + 1];
                                    if constexpr (kWords > 1) {
                                        p0 += high[j][n][2 * h];
                                        p1 += high[j][n][2 * h + 1];
                                    }
                                    acc[j][n][2 * h] = fmaf(f, p0, acc[j][n][2 * h]);
                                    if constexpr (kKind != 0) acc[j][n][2 * h + 1] = fmaf(f, p1, acc[j][n][2 * h + 1]);
                                }
                    };
                    auto groups = [&](auto kind) {
                        const int left = n_groups - ks * kGroups;
                        if (left >= kGroups) {
#pragma unroll
                            for (int q = 0; q < kGroups; ++q) group(q, kind);
                        } else {
#pragma unroll
                            for (int q = 0; q < kGroups; ++q)
                                if (q < left) group(q, kind);
                        }
                    };
                    if (nc == 1) groups(std::integral_constant<int, 0>{});
                    else if (NT == 1 || nt == 1) groups(std::integral_constant<int, 1>{});
                    else groups(std::integral_constant<int, NT>{});
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                // join the two sets of stages: one gives its sums (two buffers, so one barrier a unit)
                float* sums_of = join + turn * kJoin + 32 * rw + lane;
                if (kh == 1)
#pragma unroll
                    for (int i = 0; i < kTiles * 4 * NT; ++i) sums_of[i * 32 * kRowWarps] = acc[i / (4 * NT)][(i >> 2) % NT][i & 3];
                computing_sync();
                if (kh == 1 || *abort_flag) continue;
#pragma unroll
                for (int i = 0; i < kTiles * 4 * NT; ++i) acc[i / (4 * NT)][(i >> 2) % NT][i & 3] += sums_of[i * 32 * kRowWarps];
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = 8 * n + 2 * t + i, ya = b * kUnit + ra[j];
                            if (c >= nc) continue;
                            const float v0 = acc[j][n][i] * unscale[c], v1 = acc[j][n][2 + i] * unscale[c];
                            const int64_t at = (int64_t)(lo + base + c) * a.y_stride + ya;
                            if constexpr (UP) {
                                if (ya < a.N) store_value(a.y, a.y_type, at, silu_times<false>(v0, v1));
                            } else {
                                if (ya < a.N) store_value(a.y, a.y_type, at, v0);
                                if (ya + 8 < a.N) store_value(a.y, a.y_type, at + 8, v1);
                            }
                        }
            }
        }
    }
    if (bad && a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
    if (warp > kWarps && lane == 0) done[warp - kWarps - 1] = last;
    __syncthreads();
    if (tid == kWarps * 32 && *abort_flag) {
        // codes that no warp waited for may still be in flight: complete the phases of the steps that each stage was last
        // filled for, on behalf of the scale warps that have not arrived for them, and wait, within the limit, for the
        // bytes.  The scale warps have waited for their own copies.
        const int first = max(0, n_issued - kStages);
        for (int i = first; i < n_issued; ++i)
            if (done[i % kScaleWarps] <= i)
                for (int l = 0; l < 32; ++l) mbar_arrive(&full[i % kStages]);
        const uint64_t t0 = gtime();
        for (int i = first; i < n_issued; ++i)
            while (!mbar_test(&full[i % kStages], (i / kStages) & 1) && gtime() - t0 < p.wait_ns) {}
        if (a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_TIMEOUT);
    }
    __syncthreads();
}

template <int G, bool UP, int NT>
size_t fixed_bytes(const RowsArgs& a) {
    return 1024 + (size_t)kStages * (kStageBytes + stage_scales<G>()) + 8 * NT * 4 + 2 * kTiles * 4 * NT * 32 * kRowWarps * 4 +
           kWarps * 4 + (2 * kStages + 2) * 8 + 80 +
           (size_t)(a.E + 1) * 4 + (size_t)a.E * 2;
}

template <int G, bool UP, int NT, bool SCALE_BF16>
cudaError_t launch_as(const RowsArgs& a, cudaStream_t s) {
    W4Params p{};
    p.a = a;
    const int n_ks = (a.K + kStageK - 1) / kStageK;
    p.x_stride = n_ks * kStageK * 2 + 64;               // (8 rows' 16-byte reads fall into different banks)
    const size_t fixed = fixed_bytes<G, UP, NT>(a);
    const int most = a.offsets ? a.P / a.k : a.P;
    p.cols = (int)(((size_t)kSmemMax - fixed) / p.x_stride);
    if (p.cols > 8 * NT) p.cols = 8 * NT;
    if (p.cols > most) p.cols = most;
    if (fixed > (size_t)kSmemMax || p.cols < 1) return cudaErrorInvalidValue;    // (n_in is limited for this)
    const cuuint64_t dims[3] = {(cuuint64_t)a.K / 2, (cuuint64_t)a.E * a.N, 1}, strides[2] = {(cuuint64_t)a.K / 2, 0};
    if (!encode_map(&p.tw0, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w0, dims, strides, 128, UP ? 64 : 128) ||
        (UP && !encode_map(&p.tw1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w1, dims, strides, 128, 64)))
        return cudaErrorInvalidValue;
    p.vec = a.K % kStageK == 0 && (((uintptr_t)a.s0 | (uintptr_t)a.s1) & 15) == 0 && (((uintptr_t)a.z0 | (uintptr_t)a.z1) & 7) == 0 &&
            (G < 128 || (int64_t)a.E * a.N * (a.K / G) % 4 == 0);    // (copies of 4 zero points stay inside)
    const WaitCfg wc = wait_cfg();
    p.wait_ns = wc.limit_ns; p.stall = wc.stall;
    static std::atomic<uint64_t> ready;
    int sms = 0;
    const void* fn = (const void*)w4_kernel<G, UP, NT, SCALE_BF16>;
    cudaError_t err = prepare_kernel(fn, kSmemMax, ready, &sms);
    if (err != cudaSuccess) return err;
    constexpr int kUnit = UP ? 64 : 128;
    const int64_t units = (int64_t)(a.offsets && a.E < a.P ? a.E : a.offsets ? a.P : 1) * ((a.N + kUnit - 1) / kUnit);
    void* args[] = {&p};
    const size_t smem = fixed + (size_t)p.cols * p.x_stride;
    return launch_early(fn, dim3((unsigned)(units < sms ? units : sms)), kThreads, smem, s, args);
}

template <int G, bool UP, int NT>
cudaError_t launch(const RowsArgs& a, cudaStream_t s) {
    return a.s_bf16 ? launch_as<G, UP, NT, true>(a, s) : launch_as<G, UP, NT, false>(a, s);
}

template <int G>
cudaError_t launch_g(const RowsArgs& a, cudaStream_t s) {
    // 16 rows at once where a token batch has more than 8 and they fit beside the ring
    const int n_ks = (a.K + kStageK - 1) / kStageK;
    const bool two = (a.offsets ? a.P / a.k : a.P) > 8 &&
                     fixed_bytes<G, true, 2>(a) + 16 * ((size_t)n_ks * kStageK * 2 + 64) <= (size_t)kSmemMax;
    if (a.w1) return two ? launch<G, true, 2>(a, s) : launch<G, true, 1>(a, s);
    return two ? launch<G, false, 2>(a, s) : launch<G, false, 1>(a, s);
}

}  // namespace

cudaError_t launch_w4(const RowsArgs& a, cudaStream_t s) {
    if (a.P <= 0) return cudaSuccess;
    if (a.group == 128) return launch_g<128>(a, s);
    if (a.group == 64) return launch_g<64>(a, s);
    return launch_g<32>(a, s);
}

}  // namespace moe
