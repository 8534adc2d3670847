// w4.cu -- products of a few rows per expert with 4-bit weights and group scales.
//
//   y[i, n] = sum_g s[n, g] * (sum_{c in g} q[n, c] v_i[c] - z[n, g] * sum_{c in g} v_i[c])
// (and silu(W v) * (W_up v) of two such products), v_i = x[sorted_pairs[i] / k] or x[i].
//
// Bound: the bytes of the codes and scales; next to that the instructions that turn a code into an
// operand.  Both shape the kernel:
// - Codes come by TMA into a ring of shared memory (128 rows x 256 codes a stage, six stages in flight
//   a SM), so that the reads in flight do not depend on registers.  128-byte swizzled rows make the
//   warps' reads of 8 rows x 16 bytes free of bank conflicts.
// - The products run on the warps' m16n8k16 instruction, weights as the 16-row operand (8 rows of W
//   and the same 8 of W_up when gated, so that both halves of an output meet in one thread), up to 8 rows of
//   x as its columns.  Its sum over c may run in any order, so codes are used in the order in which they lie: a
//   32-bit word gives four operand registers by one mask each (and one shift): nibble j and j + 4 become the
//   16-bit halves.  A masked nibble q, read as fp16, is the subnormal q * 2^-24 (nibbles 0, 2) or q * 2^-20
//   (1, 3: x is stored with 1/16 there), exactly; the instruction takes subnormals exactly.  Five
//   instructions a word instead of the eleven of an exact integer-to-float conversion and subtraction.
// - The zero point is taken off the group's sum, with the group's sum of x: z is at most 15, so that costs at
//   most one bit of the fp32 sum.  Sums are fp32; the scale is applied to them in fp32.
// - x is staged once per expert: scaled by a power of two of its row's largest magnitude into fp16 (a
//   value keeps all its bits down to 2^-27 of the largest; what is lost below is less than the
//   rounding of the fp32 sum), in the word order of the codes, with the sums of each group.
// 8 computing warps of 16 weight rows each, one loading warp; a CTA per SM takes an even share of the
// (expert, 128 rows) units.
#include "internal.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);
constexpr int kStages = 6, kStageBytes = 128 * 128, kStageK = 256;
constexpr int kSmemMax = 227 * 1024;

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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void store_y(void* y, int type, int64_t i, float v) {
    if (type == MOE_F32) reinterpret_cast<float*>(y)[i] = v;
    else if (type == MOE_BF16) reinterpret_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(y)[i] = __float2half_rn(v);
}
__device__ __forceinline__ void computing_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// A stage's share of a row's scales and zero points, 256 / G of each.
template <int G>
struct Scales {
    static constexpr int kN = kStageK / G;
    uint32_t s[kN / 2], z[(kN + 3) / 4];
};
// Those of groups g0 .. of row `row` (of all experts' rows); zeros past the row's end.  vec: rows hold a
// whole number of stages and start on their size.
template <int G>
__device__ __forceinline__ void load_scales(Scales<G>& o, const void* s, const uint8_t* z, int64_t row, int g0, int n_groups,
                                            bool vec) {
    constexpr int kN = Scales<G>::kN;
    const uint16_t* sp = static_cast<const uint16_t*>(s) + row * n_groups + g0;
    const uint8_t* zp = z ? z + row * n_groups + g0 : nullptr;
#pragma unroll
    for (int i = 0; i < (kN + 3) / 4; ++i) o.z[i] = 0x08080808u;
    if (vec) {
        if constexpr (G == 32) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp));
            o.s[0] = v.x; o.s[1] = v.y; o.s[2] = v.z; o.s[3] = v.w;
            if (zp) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(zp));
                o.z[0] = w.x; o.z[1] = w.y;
            }
        } else if constexpr (G == 64) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
            o.s[0] = v.x; o.s[1] = v.y;
            if (zp) o.z[0] = __ldg(reinterpret_cast<const uint32_t*>(zp));
        } else {
            o.s[0] = __ldg(reinterpret_cast<const uint32_t*>(sp));
            if (zp) o.z[0] = __ldg(reinterpret_cast<const uint16_t*>(zp));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) o.s[i] = 0u;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (g0 + i < n_groups) {
            o.s[i >> 1] |= (uint32_t)__ldg(sp + i) << (16 * (i & 1));
            if (zp) o.z[i >> 2] = (o.z[i >> 2] & ~(0xFFu << (8 * (i & 3)))) | (uint32_t)__ldg(zp + i) << (8 * (i & 3));
        }
}

template <int G, bool UP, int NT>
__global__ void __launch_bounds__(kThreads, 1) w4_kernel(const __grid_constant__ W4Params p) {
    constexpr int kCols = 8 * NT, kUnit = UP ? 64 : 128;   // outputs of a unit
    constexpr int kGroups = kStageK / G;                   // groups of a stage
    const RowsArgs& a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int n_groups = a.K / G, n_ks = (a.K + kStageK - 1) / kStageK;
    uint8_t* xs = ring_base + kStages * kStageBytes;       // staged x: p.cols rows, p.x_stride bytes apart
    float* sums = reinterpret_cast<float*>(xs + (size_t)p.cols * p.x_stride);   // [n_ks * kGroups][kCols]
    float* unscale = sums + (size_t)n_ks * kGroups * kCols;                     // [kCols] the rows' powers of two
    uint64_t* full = reinterpret_cast<uint64_t*>(unscale + kCols);
    uint64_t* empty = full + kStages;
    uint64_t* never = empty + kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
    int* cnt = reinterpret_cast<int*>(never + 2);          // [16]
    int* off = cnt + 16;                                   // [E + 1]
    uint16_t* expert = reinterpret_cast<uint16_t*>(off + a.E + 1);   // [E] those with rows

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], kWarps); }
        mbar_init(never, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
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
        int base = n_active;
        for (int w = 0; w <= kWarps; ++w) {
            if (w < warp) base += cnt[w];
            n_active += cnt[w];
        }
        if (has) expert[base + __popc(m & ((1u << lane) - 1u))] = (uint16_t)e;
        __syncthreads();
    }
    const int n_blk = (a.N + kUnit - 1) / kUnit;
    const int64_t units = (int64_t)n_active * n_blk;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;

    // Bounded wait; after a wait has run out every wait returns at once and the loops run to their
    // ends without waiting, loading or storing, so that the CTA's barriers stay matched.
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
    int s = 0, n_issued = 0;
    uint32_t ph = 0;
    for (int64_t u = u0; u < u1;) {
        // the units of one expert
        const int e = expert[u / n_blk], b0 = (int)(u % n_blk);
        const int b1 = (int)min((int64_t)n_blk, b0 + (u1 - u));
        const int lo = off[e], rows = off[e + 1] - lo;
        u += b1 - b0;
        for (int base = 0; base < rows; base += p.cols) {
            if (warp == kWarps) {
                // ======================= loads =======================
                for (int b = b0; b < b1; ++b)
                    for (int ks = 0; ks < n_ks; ++ks) {
                        wait(&empty[s], ph ^ 1);
                        __syncwarp();
                        if (lane == 0 && !*abort_flag) {
                            mbar_expect_tx(&full[s], kStageBytes);
                            uint8_t* dst = ring_base + s * kStageBytes;
                            const int row = e * a.N + b * kUnit;
                            tma_load_2d(dst, &p.tw0, ks * 128, row, &full[s]);
                            if constexpr (UP) tma_load_2d(dst + 8192, &p.tw1, ks * 128, row, &full[s]);
                            mbar_arrive(&full[s]);
                            ++n_issued;
                        }
                        if (++s == kStages) { s = 0; ph ^= 1; }
                    }
                continue;
            }
            // ======================= staging of x =======================
            const int nc = min(p.cols, rows - base);
            computing_sync();                            // the rows before have been used
            for (int c = warp; c < nc; c += kWarps) {
                int64_t row = lo + base + c;
                if (a.sorted_pairs) {
                    const int pair = __ldg(a.sorted_pairs + row);
                    const bool in = (uint32_t)pair < (uint32_t)a.P;
                    bad |= !in;
                    row = in ? pair / a.k : 0;
                }
                const uint16_t* src = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
                auto load = [&](int i, float (&v)[8]) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + i));
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
                float most = 0.f;
                for (int i = 8 * lane; i < a.K; i += 256) {
                    float v[8];
                    load(i, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[j]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                // the largest becomes 2^14 .. 2^15 (a row of zeros, and one that is not finite, stay)
                const int mexp = (int)(__float_as_uint(most) >> 23);
                const int ex = mexp == 0 || mexp == 255 ? 0 : min(max(mexp - 127 - 14, -120), 113);
                const float scale = __int_as_float((127 - ex) << 23);
                if (lane == 0) unscale[c] = __int_as_float((127 + ex) << 23);
                for (int i = 8 * lane; i < n_ks * kStageK; i += 256) {
                    float v[8] = {};
                    if (i < a.K) load(i, v);
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[j] *= scale;
                        sum += v[j];
                    }
                    const __half2 h0 = __floats2half2_rn(v[0], v[4]), h1 = __floats2half2_rn(v[1] * 0.0625f, v[5] * 0.0625f);
                    const __half2 h2 = __floats2half2_rn(v[2], v[6]), h3 = __floats2half2_rn(v[3] * 0.0625f, v[7] * 0.0625f);
                    *reinterpret_cast<uint4*>(xs + (size_t)c * p.x_stride + 2 * i) =
                        make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                                   *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3));
#pragma unroll
                    for (int o = 1; o < G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane % (G / 8) == 0) sums[(i / G) * kCols + c] = sum;
                }
            }
            computing_sync();
            // ======================= products =======================
            const int nt = (nc + 7) / 8;
            const uint8_t* xc[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xc[n] = 8 * n + g < nc ? xs + (size_t)(8 * n + g) * p.x_stride : nullptr;
            const int ra = UP ? 8 * warp + g : 16 * warp + g, rb = UP ? 64 + 8 * warp + g : 16 * warp + 8 + g;   // in the stage
            const int ya = ra, yb = UP ? ra : rb;          // outputs of the two rows, in the unit
            // scales of the two rows, two stages ahead
            Scales<G> sa[3], sb[3];
            int pb = b0, pk = 0;
            auto ahead = [&](Scales<G>& qa, Scales<G>& qb) {
                if (pb < b1) {
                    const int64_t r0 = (int64_t)e * a.N + min(pb * kUnit + ya, a.N - 1);
                    const int64_t r1 = (int64_t)e * a.N + min(pb * kUnit + yb, a.N - 1);
                    load_scales<G>(qa, a.s0, a.z0, r0, pk * kGroups, n_groups, p.vec);
                    load_scales<G>(qb, UP ? a.s1 : a.s0, UP ? a.z1 : a.z0, r1, pk * kGroups, n_groups, p.vec);
                    if (++pk == n_ks) { pk = 0; ++pb; }
                }
            };
            ahead(sa[0], sb[0]);
            ahead(sa[1], sb[1]);
            for (int b = b0; b < b1; ++b) {
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
                for (int ks = 0; ks < n_ks; ++ks) {
                    ahead(sa[2], sb[2]);
                    const bool stalled = p.stall && u - b1 + b == u0 && ks == 0;      // (test setting)
                    wait(stalled ? never : &full[s], stalled ? 0u : ph);
                    const uint8_t* wa = ring_base + s * kStageBytes + ra * 128;
                    const uint8_t* wb = ring_base + s * kStageBytes + rb * 128;
                    const int left = min(kGroups, n_groups - ks * kGroups);
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        if (q >= left) break;
                        // this lane's quarter of the group's codes, of both rows
                        constexpr int kWords = G / 32;
                        uint32_t va[kWords], vb[kWords];
                        const int byte = q * (G / 2) + t * (G / 8);
                        const int o = (((byte >> 4) ^ g) << 4) + (byte & 15);
                        if constexpr (G == 128) {
                            const uint4 x0 = *reinterpret_cast<const uint4*>(wa + o), x1 = *reinterpret_cast<const uint4*>(wb + o);
                            va[0] = x0.x; va[1] = x0.y; va[2] = x0.z; va[3] = x0.w;
                            vb[0] = x1.x; vb[1] = x1.y; vb[2] = x1.z; vb[3] = x1.w;
                        } else if constexpr (G == 64) {
                            const uint2 x0 = *reinterpret_cast<const uint2*>(wa + o), x1 = *reinterpret_cast<const uint2*>(wb + o);
                            va[0] = x0.x; va[1] = x0.y;
                            vb[0] = x1.x; vb[1] = x1.y;
                        } else {
                            va[0] = *reinterpret_cast<const uint32_t*>(wa + o);
                            vb[0] = *reinterpret_cast<const uint32_t*>(wb + o);
                        }
                        float part[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
#pragma unroll
                        for (int w = 0; w < kWords; ++w) {
                            const uint32_t a8 = va[w] >> 8, b8 = vb[w] >> 8;
                            const int xo = 2 * (ks * kStageK + q * G + t * (G / 4) + 8 * w);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (n >= nt) break;
                                const uint4 x = xc[n] ? *reinterpret_cast<const uint4*>(xc[n] + xo) : make_uint4(0u, 0u, 0u, 0u);
                                mma_f16_16816(part[n], va[w] & 0x000F000Fu, vb[w] & 0x000F000Fu, va[w] & 0x00F000F0u,
                                              vb[w] & 0x00F000F0u, x.x, x.y);
                                mma_f16_16816(part[n], a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u, b8 & 0x00F000F0u,
                                              x.z, x.w);
                            }
                        }
                        const uint32_t ha = sa[0].s[q >> 1] >> (16 * (q & 1)), hb = sb[0].s[q >> 1] >> (16 * (q & 1));
                        float fa, fb;
                        if (a.s_bf16) {
                            fa = __uint_as_float(ha << 16);
                            fb = __uint_as_float(hb << 16);
                        } else {
                            fa = __half2float(__ushort_as_half((unsigned short)ha));
                            fb = __half2float(__ushort_as_half((unsigned short)hb));
                        }
                        // -z * 2^-24, exactly: 2^23 + z as a float's bits, times -2^-24, plus 1/2
                        const float za = fmaf(__uint_as_float(0x4B000000u | ((sa[0].z[q >> 2] >> (8 * (q & 3))) & 15u)), -0x1p-24f, 0.5f);
                        const float zb = fmaf(__uint_as_float(0x4B000000u | ((sb[0].z[q >> 2] >> (8 * (q & 3))) & 15u)), -0x1p-24f, 0.5f);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n >= nt) break;
                            const float2 xsum = *reinterpret_cast<const float2*>(sums + (size_t)(ks * kGroups + q) * kCols + 8 * n + 2 * t);
                            acc[n][0] = fmaf(fa, fmaf(za, xsum.x, part[n][0]), acc[n][0]);
                            acc[n][1] = fmaf(fa, fmaf(za, xsum.y, part[n][1]), acc[n][1]);
                            acc[n][2] = fmaf(fb, fmaf(zb, xsum.x, part[n][2]), acc[n][2]);
                            acc[n][3] = fmaf(fb, fmaf(zb, xsum.y, part[n][3]), acc[n][3]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    if (++s == kStages) { s = 0; ph ^= 1; }
                    sa[0] = sa[1]; sb[0] = sb[1];
                    sa[1] = sa[2]; sb[1] = sb[2];
                }
                if (*abort_flag) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = 8 * n + 2 * t + i;
                        if (c >= nc) continue;
                        const float v0 = acc[n][i] * 0x1p24f * unscale[c], v1 = acc[n][2 + i] * 0x1p24f * unscale[c];
                        const int64_t at = (int64_t)(lo + base + c) * a.y_stride + b * kUnit;
                        if constexpr (UP) {
                            if (b * kUnit + ya < a.N) store_y(a.y, a.y_type, at + ya, v0 / (1.0f + expf(-v0)) * v1);
                        } else {
                            if (b * kUnit + ya < a.N) store_y(a.y, a.y_type, at + ya, v0);
                            if (b * kUnit + yb < a.N) store_y(a.y, a.y_type, at + yb, v1);
                        }
                    }
            }
        }
    }
    if (bad && a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
    __syncthreads();
    if (tid == kWarps * 32 && *abort_flag) {
        // copies that no warp waited for may still be in flight: wait (within the limit) for their stages
        for (int i = 0; i < min(n_issued, kStages); ++i) {
            const int step = n_issued - 1 - i;
            const uint64_t t0 = gtime();
            while (!mbar_test(&full[step % kStages], (step / kStages) & 1) && gtime() - t0 < p.wait_ns) {}
        }
        if (a.status) atomicCAS(a.status, (int)MOE_OK, (int)MOE_ERR_TIMEOUT);
    }
    __syncthreads();
}

template <int G, bool UP, int NT>
size_t fixed_bytes(const RowsArgs& a, int n_ks) {
    return 1024 + (size_t)kStages * kStageBytes + (size_t)n_ks * (kStageK / G) * 8 * NT * 4 + 8 * NT * 4 + (2 * kStages + 2) * 8 + 64 +
           (size_t)(a.E + 1) * 4 + (size_t)a.E * 2;
}

template <int G, bool UP, int NT>
cudaError_t launch(const RowsArgs& a, cudaStream_t s) {
    W4Params p{};
    p.a = a;
    const int n_ks = (a.K + kStageK - 1) / kStageK;
    p.x_stride = n_ks * kStageK * 2 + 64;               // (8 rows' 16-byte reads fall into different banks)
    const size_t fixed = fixed_bytes<G, UP, NT>(a, n_ks);
    const int most = a.offsets ? a.P / a.k : a.P;
    p.cols = (int)(((size_t)kSmemMax - fixed) / p.x_stride);
    if (p.cols > 8 * NT) p.cols = 8 * NT;
    if (p.cols > most) p.cols = most;
    if (fixed > (size_t)kSmemMax || p.cols < 1) return cudaErrorInvalidValue;    // (n_in is limited for this)
    const cuuint64_t dims[3] = {(cuuint64_t)a.K / 2, (cuuint64_t)a.E * a.N, 1}, strides[2] = {(cuuint64_t)a.K / 2, 0};
    if (!encode_map(&p.tw0, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w0, dims, strides, 128, UP ? 64 : 128) ||
        (UP && !encode_map(&p.tw1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w1, dims, strides, 128, 64)))
        return cudaErrorInvalidValue;
    p.vec = a.K % kStageK == 0 && (((uintptr_t)a.s0 | (uintptr_t)a.s1) & 15) == 0 && (((uintptr_t)a.z0 | (uintptr_t)a.z1) & 7) == 0;
    const WaitCfg wc = wait_cfg();
    p.wait_ns = wc.limit_ns; p.stall = wc.stall;
    static std::atomic<uint64_t> ready;
    int sms = 0;
    const void* fn = (const void*)w4_kernel<G, UP, NT>;
    cudaError_t err = prepare_kernel(fn, kSmemMax, ready, &sms);
    if (err != cudaSuccess) return err;
    constexpr int kUnit = UP ? 64 : 128;
    const int64_t units = (int64_t)(a.offsets && a.E < a.P ? a.E : a.offsets ? a.P : 1) * ((a.N + kUnit - 1) / kUnit);
    void* args[] = {&p};
    const size_t smem = fixed + (size_t)p.cols * p.x_stride;
    err = cudaLaunchKernel(fn, dim3((unsigned)(units < sms ? units : sms)), dim3(kThreads), args, smem, s);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <int G>
cudaError_t launch_g(const RowsArgs& a, cudaStream_t s) {
    // 16 rows at once where a token batch has more than 8 and they fit beside the ring
    const int n_ks = (a.K + kStageK - 1) / kStageK;
    const bool two = (a.offsets ? a.P / a.k : a.P) > 8 &&
                     fixed_bytes<G, true, 2>(a, n_ks) + 16 * ((size_t)n_ks * kStageK * 2 + 64) <= (size_t)kSmemMax;
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
