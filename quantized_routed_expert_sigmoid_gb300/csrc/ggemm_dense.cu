// ggemm_dense.cu -- grouped products over bf16 / fp16 expert weights on the 5th-generation tensor
// cores, for more rows than the streaming kernel of rows.cu can carry.
//
//   y[i, n] = sum_c W[e][n, c] v_i[c],  or  silu(W v) * (W_up v),   v_i = x[sorted_pairs[i] / k] or x[i]
//
// A pair of CTAs (cta_group::2) computes one tile: 256 weight rows (M) by up to 256 rows of x of one
// expert (N, a multiple of 32), c in steps of 64.  The weights are the M operand because their extent
// is always large: an expert with 3 rows pays for 32 columns, not for 128 rows of M.  Each CTA
// loads 128 weight rows and half of the columns (32 KB a step) and keeps the accumulators of its 128
// weight rows in TMEM, so a weight element is read from L2 once per 256 rows of x and an x element
// once per 256 outputs.  With a one-CTA tile of 128 x 256 a step loads 48 KB per SM for the same number of
// flops per SM, more than L2 delivers at the tensor cores' rate.
// Gated pair: the 128 M rows of a CTA are 64 rows of W and the same 64 rows of W_up, so that both
// halves of an output lie in one CTA's TMEM (lanes r and 64 + r); two epilogue warps trade
// halves of their columns through shared memory and each computes silu(g) u for its half.
// [in][out] weights enter as an MN-major operand (the descriptor's transpose bit): the same boxes
// with their axes exchanged, no transposed copy.
//
// Warps: 0 loads (TMA: two 64 x 64 weight boxes, and the x rows in place as 16-row boxes), 1 issues the
// MMAs (in the first CTA of the pair) and owns TMEM, 2 and 3 copy the x rows that the pairs name (cp.async,
// 16 bytes a thread, four steps in flight; TMA's four-row gathers took 70 clocks each, 594 us for the
// gated half of 4096 tokens), 4..11 are the epilogue (two accumulators of 256 columns: one is
// read out while the next tile runs).  Persistent:
// a pair takes every (pairs of CTAs)-th tile of the list that the offsets define, each warp role finding its
// tiles by itself.  Every wait is bounded; a wait that runs out is reported (MOE_ERR_TIMEOUT), the copies in flight
// are waited for (bounded), TMEM is freed and the kernel returns.
#include <atomic>
#include <cuda.h>   // CUtensorMap and its enums (the encoder is fetched from the driver at run time)

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kStages = 6, kStepK = 64, kMaxN = 256;
constexpr int kABytes = 128 * 128, kBBytes = 128 * 128, kStageBytes = kABytes + kBBytes;
constexpr int kThreads = 384, kGatherWarp0 = 2, kGatherWarps = 2, kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kGatherAhead = 4;                          // steps a gathering thread has in flight
constexpr int kGatherRows = 128 / (4 * kGatherWarps);    // rows of a step a gathering thread copies 16 bytes of
constexpr int kExchBytes = 4 * 2 * 2 * 8 * 32 * 4;       // [warp pair][buffer][half][column][lane] floats
constexpr uint32_t kTmemCols = 512;

struct DenseParams {
    CUtensorMap tw0, tw1;        // W, W_up: [E][rows][cols], boxes of 64 x 64
    CUtensorMap tx;              // x rows in place: boxes of 64 x 16
    const uint16_t* x;           // x rows for the gather
    int64_t x_stride;
    const int32_t* sorted_pairs; // NULL: rows in place
    const int32_t* offsets;      // NULL: one expert over all P rows
    int E, k, P, N, K;
    bool bf16, in_out;
    void* y;
    int y_type;
    int64_t y_stride;
    int32_t* status;
    uint64_t wait_ns;
    int stall;                   // test setting: the first wait of the MMA warp never completes
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The pair's barriers order copies and MMAs, which carry their own ordering; no plain loads or stores
// pass from CTA to CTA through them.  So their operations take the default scope: with release and
// acquire at cluster scope every step of the pipeline waited about 0.5 us for its arrival.
// Shared address of the pair's first CTA (the one that issues the MMAs) for an address of this one.
__device__ __forceinline__ uint32_t in_leader(uint32_t a) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t in_peer(uint32_t a) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_tx_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Bounded wait of a whole warp on a barrier that either CTA of the pair arrives on: false on every lane
// after limit_ns (raising abort_flag) or when another warp of this CTA has raised it.
__device__ __forceinline__ bool wait_cluster(uint64_t* b, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
    bool ok = mbar_test(b, parity);
    if (!ok) {
        const uint64_t t0 = gtime();
        while (!(ok = mbar_test(b, parity))) {
            if (*abort_flag) break;
            if (gtime() - t0 > limit_ns) { *abort_flag = 1; break; }
        }
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void drain_wait(uint64_t* b, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = gtime();
    while (!mbar_test(b, parity))
        if (gtime() - t0 > limit_ns) return;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// All MMAs issued so far arrive on this barrier of both CTAs when they are done.
__device__ __forceinline__ void commit_pair(uint64_t* b) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(b)),
        "h"((uint16_t)3)
        : "memory");
}
// MN-major operand, 128-byte swizzle: 64-element blocks along M 8192 bytes apart, groups of 8 c 1024.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
        "%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
// True on every thread of the named barrier when it is true on all of them.
__device__ __forceinline__ bool all_of(int barrier, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(barrier), "r"(threads), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void named_sync(int barrier, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}

__device__ __forceinline__ void store_out(void* y, int type, int64_t i, float v) {
    if (type == MOE_F32) reinterpret_cast<float*>(y)[i] = v;
    else if (type == MOE_BF16) reinterpret_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(y)[i] = __float2half_rn(v);
}

struct Tile {
    int e, mb, tok0, ntok, nh;   // expert, block of M rows, first sorted position, rows, columns per CTA
};
// Tile t of the list: experts in order, their rows in even blocks of at most 256, blocks of M rows fastest
// (the pairs that run at one time share the rows of x and walk through one expert's weights).
__device__ __forceinline__ bool tile_at(const int* off, const int* tb0, int E, int n_mb, int t, Tile& ti) {
    const int tb = t / n_mb;
    if (tb >= tb0[E]) return false;
    int lo = 0, hi = E;                                  // tb0[lo] <= tb < tb0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tb0[mid] <= tb) lo = mid; else hi = mid;
    }
    const int cnt = off[lo + 1] - off[lo], nb = tb0[lo + 1] - tb0[lo], blk = tb - tb0[lo];
    const int per = ((cnt + nb - 1) / nb + 31) & ~31;    // (nb - 1) * per < cnt, as per <= 256 < cnt / (nb - 1)
    ti.e = lo;
    ti.mb = t - tb * n_mb;
    ti.tok0 = off[lo] + blk * per;
    ti.ntok = min(per, cnt - blk * per);
    ti.nh = ((ti.ntok + 31) & ~31) >> 1;
    return true;
}

template <bool UP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) grouped_dense_kernel(const __grid_constant__ DenseParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float* exch = reinterpret_cast<float*>(smem + kStages * kStageBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + kExchBytes);   // first CTA's: both CTAs' bytes
    uint64_t* empty = full + kStages;                    // the step's MMAs are done
    uint64_t* accf = empty + kStages;                    // [2]: accumulator complete
    uint64_t* accr = accf + 2;                           // [2]: accumulator read out (both CTAs' warps)
    uint64_t* drain = accr + 2;
    uint64_t* never = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* done = reinterpret_cast<int*>(tmem_slot + 2);   // steps that warps 0, 2 and 3 have arrived for
    int* scan = reinterpret_cast<int*>(tmem_slot + 6);   // [16]
    int* off = scan + 16;                                // [E + 1] offsets, clamped and in order
    int* tb0 = off + p.E + 1;                            // [E + 1] blocks of rows before each expert

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t cta = cta_rank();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], p.sorted_pairs ? 2 + 2 * kGatherWarps : 2); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&accf[i], 1); mbar_init(&accr[i], 2 * kEpiWarps); }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        for (int i = 0; i < 1 + kGatherWarps; ++i) done[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // ---- the list of row blocks, from the offsets (clamped into 0..P and into order)
    bool bad = false;
    for (int i = tid; i <= p.E; i += kThreads) {
        const int o = p.offsets ? __ldg(p.offsets + i) : (i ? p.P : 0);
        bad |= o < 0 || o > p.P || (i > 0 && p.offsets && __ldg(p.offsets + i - 1) > o);
        off[i] = min(max(o, 0), p.P);
    }
    __syncthreads();
    {
        // thread t: experts t * per .. of a scan over the whole block
        const int per = (p.E + kThreads - 1) / kThreads, e0 = tid * per;
        int sum = 0;
        for (int i = e0; i < min(e0 + per, p.E); ++i) sum += (max(off[i + 1] - off[i], 0) + kMaxN - 1) / kMaxN;
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int base = inc - sum;
        for (int w = 0; w < warp; ++w) base += scan[w];
        for (int i = e0; i < min(e0 + per, p.E); ++i) {
            tb0[i] = base;
            base += (max(off[i + 1] - off[i], 0) + kMaxN - 1) / kMaxN;
            if (i == p.E - 1) tb0[p.E] = base;
        }
    }
    tc_before();
    __syncthreads();
    cluster_sync();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int kRowsTile = UP ? 128 : 256;            // outputs of a tile of the pair
    const int n_mb = (p.N + kRowsTile - 1) / kRowsTile;
    const int n_pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
    const int nk = (p.K + kStepK - 1) / kStepK;

    if (warp == 0) {
        // ======================= loads =======================
        const uint32_t full0 = in_leader(su32(full));
        uint32_t g = 0;
        bool ok = true;
        Tile ti;
        for (int t = first; ok && tile_at(off, tb0, p.E, n_mb, t, ti); t += n_pairs) {
            const int c0 = ti.tok0 + (int)cta * ti.nh;   // this CTA's first column, as a sorted position
            const int r0 = ti.mb * kRowsTile + (int)cta * (kRowsTile / 2);
            const uint32_t bytes = kABytes + (p.sorted_pairs ? 0 : ti.nh * 128);
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const int s = g % kStages;
                if (g >= kStages && !wait_cluster(&empty[s], (g / kStages - 1) & 1, abort_flag, p.wait_ns)) { ok = false; break; }
                const uint32_t bar = full0 + 8 * s;
                const uint32_t a = su32(smem + s * kStageBytes), b = a + kABytes;
                if (lane == 0) {
                    arrive_tx_cluster(bar, bytes);
                    const int c = kb * kStepK;
                    if (p.in_out) {
                        tma_3d(a, &p.tw0, r0, c, ti.e, bar);
                        tma_3d(a + 8192, UP ? &p.tw1 : &p.tw0, UP ? r0 : r0 + 64, c, ti.e, bar);
                    } else {
                        tma_3d(a, &p.tw0, c, r0, ti.e, bar);
                        tma_3d(a + 8192, UP ? &p.tw1 : &p.tw0, c, UP ? r0 : r0 + 64, ti.e, bar);
                    }
                    done[0] = (int)g + 1;
                }
                if (!p.sorted_pairs && 16 * lane < ti.nh)
                    tma_2d(b + 2048 * lane, &p.tx, kb * kStepK, c0 + 16 * lane, bar);
                __syncwarp();
            }
        }
        // the last steps' arrivals on this CTA's barriers have landed before it may leave
        if (ok)
            for (uint32_t s = g > kStages ? g - kStages : 0; s < g; ++s)
                if (!wait_cluster(&empty[s % kStages], (s / kStages) & 1, abort_flag, p.wait_ns)) break;
    } else if (warp == 1 && cta == 0) {
        // ======================= MMA issue =======================
        uint32_t g = 0;
        int j = 0;
        bool ok = true;
        Tile ti;
        for (int t = first; ok && tile_at(off, tb0, p.E, n_mb, t, ti); t += n_pairs, ++j) {
            const uint32_t idesc = idesc_mma(256, 2 * ti.nh, p.bf16) | (p.in_out ? 1u << 15 : 0u);
            const int b = j & 1;
            if (j >= 2 && !wait_cluster(&accr[b], ((j >> 1) - 1) & 1, abort_flag, p.wait_ns)) break;
            tc_after();
            const uint32_t acc = tmem + (uint32_t)b * kMaxN;
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const int s = g % kStages;
                uint64_t* fb = p.stall && g == 0 ? never : &full[s];         // (test stall)
                if (!wait_cluster(fb, fb == never ? 0u : (g / kStages) & 1, abort_flag, p.wait_ns)) { ok = false; break; }
                tc_after();
                if (lane == 0) {
                    const uint32_t a0 = su32(smem + s * kStageBytes), b0 = a0 + kABytes;
#pragma unroll
                    for (int kk = 0; kk < kStepK / 16; ++kk)
                        mma_pair(acc, p.in_out ? sdesc_mn(a0 + 2048 * kk) : sdesc(a0 + 32 * kk), sdesc(b0 + 32 * kk), idesc,
                                 (kb | kk) != 0);
                    commit_pair(&empty[s]);
                    if (kb == nk - 1) commit_pair(&accf[b]);
                }
                __syncwarp();
            }
        }
        // every MMA issued has completed before TMEM is freed
        if (g > 0) {
            if (lane == 0)
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(drain))
                             : "memory");
            __syncwarp();
            drain_wait(drain, 0, p.wait_ns);
        }
    } else if (warp >= kGatherWarp0 && warp < kEpiWarp0) {
        // ======================= gathered rows of x =======================
        if (p.sorted_pairs) {
            // thread u copies chunk u % 8 of rows u / 8 + 8 * kGatherWarps * j of a step into the swizzled layout
            const int u = tid - 32 * kGatherWarp0, ch = u & 7, w = warp - kGatherWarp0;
            constexpr int kRowStep = 4 * kGatherWarps;
            const uint32_t full0 = in_leader(su32(full));
            uint32_t g = 0, arrived = 0;
            bool ok = true;
            Tile ti;
            for (int t = first; ok && tile_at(off, tb0, p.E, n_mb, t, ti); t += n_pairs) {
                const int c0 = (int)cta * ti.nh, nc = min(ti.nh, ti.ntok - c0);   // columns of this CTA that hold rows
                int row[kGatherRows];
#pragma unroll
                for (int j = 0; j < kGatherRows; ++j) {
                    const int r = (u >> 3) + kRowStep * j;
                    row[j] = 0;
                    if (r < nc) {
                        const int pair = __ldg(p.sorted_pairs + ti.tok0 + c0 + r);
                        const bool in = pair >= 0 && pair < p.P;
                        bad |= !in;
                        row[j] = in ? pair / p.k : 0;
                    }
                }
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const int s = g % kStages;
                    if (g >= kStages && !wait_cluster(&empty[s], (g / kStages - 1) & 1, abort_flag, p.wait_ns)) { ok = false; break; }
                    const int c = kb * kStepK + 8 * ch;
                    const uint32_t bytes = (uint32_t)min(max(2 * (p.K - c), 0), 16);   // zeros past the row's end
                    uint8_t* dst = smem + s * kStageBytes + kABytes;
#pragma unroll
                    for (int j = 0; j < kGatherRows; ++j) {
                        const int r = (u >> 3) + kRowStep * j;
                        if (r < nc) cp_async16(dst + swz(r, ch), p.x + row[j] * p.x_stride + (bytes ? c : 0), bytes);
                    }
                    cp_commit();
                    if (g >= kGatherAhead) {
                        cp_wait<kGatherAhead>();
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(full0 + 8 * ((g - kGatherAhead) % kStages));
                        arrived = g - kGatherAhead + 1;
                    }
                }
            }
            cp_wait_all();
            fence_async_smem();
            __syncwarp();
            for (; ok && arrived < g; ++arrived)
                if (lane == 0) arrive_cluster(full0 + 8 * (arrived % kStages));
            if (lane == 0) done[1 + w] = (int)arrived;
        }
    } else if (warp >= kEpiWarp0) {
        // ======================= epilogue =======================
        // warp w reads TMEM lanes 32 (w % 4).. and half of the columns (groups of 32, every other one)
        const int q = warp & 3, side = (warp - kEpiWarp0) >> 2;
        const uint32_t accr0 = in_leader(su32(accr));
        const int pairbar = 1 + side * 2 + (q & 1);      // gated: warps q and q + 2 trade columns
        int j = 0, turn = 0;
        Tile ti;
        for (int t = first; tile_at(off, tb0, p.E, n_mb, t, ti); t += n_pairs, ++j) {
            const int b = j & 1;
            bool ok = wait_cluster(&accf[b], (j >> 1) & 1, abort_flag, p.wait_ns);
            // (the two warps of a trade leave together, or one would wait for the other for ever)
            if constexpr (UP) ok = all_of(pairbar, 64, ok);
            if (!ok) break;
            tc_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)b * kMaxN;
            if constexpr (UP) {
                const int row = ti.mb * kRowsTile + (int)cta * 64 + (q & 1) * 32 + lane;
                const bool is_up = q >= 2;
                for (int c0 = 16 * side; c0 < ti.ntok; c0 += 32, ++turn) {
                    uint32_t r[16];
                    tmem_ld16(acc + c0, r);
                    tmem_ld_wait();
                    // the W warp keeps columns 0..7 and gives 8..15, the W_up warp the other way round
                    float* buf = exch + (((pairbar - 1) * 2 + (turn & 1)) * 2) * 256;
                    float* mine = buf + (is_up ? 256 : 0);
                    const float* theirs = buf + (is_up ? 0 : 256);
#pragma unroll
                    for (int i = 0; i < 8; ++i) mine[i * 32 + lane] = __uint_as_float(is_up ? r[i] : r[8 + i]);
                    named_sync(pairbar, 64);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float other = theirs[i * 32 + lane];
                        const float gv = is_up ? other : __uint_as_float(r[i]);
                        const float uv = is_up ? __uint_as_float(r[8 + i]) : other;
                        const int col = c0 + (is_up ? 8 : 0) + i;
                        if (col < ti.ntok && row < p.N)
                            store_out(p.y, p.y_type, (int64_t)(ti.tok0 + col) * p.y_stride + row, gv / (1.0f + expf(-gv)) * uv);
                    }
                }
            } else {
                const int row = ti.mb * kRowsTile + (int)cta * 128 + q * 32 + lane;
                for (int c0 = 32 * side; c0 < ti.ntok; c0 += 64) {
                    uint32_t r[32];
                    tmem_ld32(acc + c0, r);
                    tmem_ld_wait();
                    if (row < p.N) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c0 + i < ti.ntok)
                                store_out(p.y, p.y_type, (int64_t)(ti.tok0 + c0 + i) * p.y_stride + row, __uint_as_float(r[i]));
                    }
                }
            }
            tc_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(accr0 + 8 * b);
        }
    }
    if (bad && p.status) atomicCAS(p.status, (int)MOE_OK, (int)MOE_ERR_DEVICE_CHECK);
    tc_before();
    __syncwarp();
    cluster_sync();                                      // both CTAs' roles have left their loops
    if (cta == 0 && tid == 0) {
        // after a timeout copies may still be in flight: complete the phases of the steps that some
        // warps have arrived for (on behalf of the others) and wait, within the limit, for the bytes
        int peer_abort;
        asm volatile("ld.volatile.shared::cluster.u32 %0, [%1];"
                     : "=r"(peer_abort)
                     : "r"(in_peer(su32(const_cast<int*>(abort_flag))))
                     : "memory");
        if (*abort_flag || peer_abort) {
            const int warps = p.sorted_pairs ? 1 + kGatherWarps : 1;
            int of[2][1 + kGatherWarps], last = 0;
            for (int i = 0; i < warps; ++i) {
                of[0][i] = done[i];
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(of[1][i]) : "r"(in_peer(su32(done + i))) : "memory");
                last = max(last, max(of[0][i], of[1][i]));
            }
            for (int c = 0; c < 2; ++c)
                for (int i = 0; i < warps; ++i)
                    for (int s = of[c][i]; s < last; ++s) mbar_arrive(&full[s % kStages]);
            for (int s = max(0, last - kStages); s < last; ++s) drain_wait(&full[s % kStages], (s / kStages) & 1, p.wait_ns);
            if (p.status) atomicCAS(p.status, (int)MOE_OK, (int)MOE_ERR_TIMEOUT);
        }
    }
    __syncwarp();
    cluster_sync();
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn got = fn.load(std::memory_order_acquire);
    if (!got) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            got = reinterpret_cast<EncodeTiledFn>(f);
            fn.store(got, std::memory_order_release);
        }
    }
    return got;
}

// 16-bit elements, boxes of 64 x box1 (x 1), 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* m, bool bf16, int rank, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
            int box1) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint32_t box[3] = {64u, (cuuint32_t)box1, 1u}, one[3] = {1u, 1u, 1u};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
              const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t smem_bytes(int E) {
    return 1024 + (size_t)kStages * kStageBytes + kExchBytes + (2 * kStages + 6) * 8 + 24 + 64 + 2 * (size_t)(E + 1) * 4;
}

}  // namespace

cudaError_t launch_grouped_dense(const RowsArgs& a, cudaStream_t s) {
    if (a.P <= 0) return cudaSuccess;
    DenseParams p{};
    const cuuint64_t rows = a.in_out ? a.K : a.N, cols = a.in_out ? a.N : a.K;
    const cuuint64_t wd[3] = {cols, rows, (cuuint64_t)a.E};
    const cuuint64_t ws[2] = {(cuuint64_t)a.row_stride * 2, a.E > 1 ? (cuuint64_t)a.expert_stride * 2
                                                                    : (cuuint64_t)a.row_stride * rows * 2};
    const cuuint64_t xd[3] = {(cuuint64_t)a.K, (cuuint64_t)a.P, 1};
    const cuuint64_t xs[2] = {(cuuint64_t)a.x_stride * 2, 0};
    if (!encode(&p.tw0, a.bf16, 3, a.w0, wd, ws, 64) || (a.w1 && !encode(&p.tw1, a.bf16, 3, a.w1, wd, ws, 64)) ||
        (!a.sorted_pairs && !encode(&p.tx, a.bf16, 2, a.x, xd, xs, 16)))
        return cudaErrorInvalidValue;
    p.x = static_cast<const uint16_t*>(a.x);
    p.x_stride = a.x_stride;
    p.sorted_pairs = a.sorted_pairs; p.offsets = a.offsets;
    p.E = a.E; p.k = a.k; p.P = a.P; p.N = a.N; p.K = a.K;
    p.bf16 = a.bf16; p.in_out = a.in_out;
    p.y = a.y; p.y_type = a.y_type; p.y_stride = a.y_stride; p.status = a.status;
    const WaitCfg wc = wait_cfg();
    p.wait_ns = wc.limit_ns; p.stall = wc.stall;
    int dev = 0, sms = 0;
    cudaError_t err;
    if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
    const void* fn = a.w1 ? (const void*)grouped_dense_kernel<true> : (const void*)grouped_dense_kernel<false>;
    static std::atomic<uint64_t> ready[2];               // devices whose function attribute is set
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!bit || !(ready[a.w1 != nullptr].load(std::memory_order_acquire) & bit)) {
        if ((err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kMaxExperts))) != cudaSuccess)
            return err;
        ready[a.w1 != nullptr].fetch_or(bit, std::memory_order_release);
    }
    // one pair per two SMs, and no more pairs than there can be tiles
    const int64_t n_mb = (a.N + (a.w1 ? 127 : 255)) / (a.w1 ? 128 : 256);
    const int64_t most = ((int64_t)a.P / kMaxN + (a.E < a.P ? a.E : a.P)) * n_mb;
    const int pairs = (int)(most < sms / 2 ? most : sms / 2);
    void* args[] = {&p};
    err = cudaLaunchKernel(fn, dim3(2 * (pairs > 0 ? pairs : 1)), dim3(kThreads), args, smem_bytes(a.E), s);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
