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
// Warps: 0 loads (TMA, as few boxes as there can be), 1 issues the MMAs (in the first CTA of the pair) and
// owns TMEM, 2, 3 and 12..17 fetch the x rows that the pairs name (TMA, four rows to a copy), 4..11 are the epilogue
// (two accumulators of 256 columns: one is read out while the next tile runs).  What is issued by one lane has
// its operands in registers that the whole warp keeps uniform: that takes 20 to 30 clocks a copy or MMA,
// lane by lane 70 to 100.  Persistent: a pair takes every (pairs of CTAs)-th tile of the order that the
// offsets define, each warp role finding its tiles by itself.  Every wait is bounded; a wait that runs out is
// reported (MOE_ERR_TIMEOUT), the copies in flight are waited for (bounded), TMEM is freed and the kernel returns.
//
// Measured (device time; bytes and flops that the products cannot do without against 6.69 TB/s and 1.95 PFLOP/s):
// 4096 tokens, 8 of 128 experts, hidden 2048, intermediate 768: gated half 172 us (206 GFLOP, 822 MB: 72 % of its
// 123 us; tensor pipe 55 %, DRAM 64 %), down with fp32 rows 116 us (90 % of 104 us, bytes); 32 tokens, down
// 57.2 us (93 %, bytes); 512 tokens, 256 experts of 2048 x 7168 stored [in][out] 1.10 ms (7.6 GB, at the copy's
// rate).  The gated half is what is left: of 171 us it took 156 without its gathers, 154 without its epilogue, 141 without
// both, and 125 with no loads at all.
#include "cluster_ptx.cuh"
#include "products.cuh"

namespace moe {
namespace {

constexpr int kStages = 6, kStepK = 64, kMaxN = 256;
constexpr int kABytes = 128 * 128, kBBytes = 128 * 128, kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;              // (a warp reads the TMEM lanes 32 (warp % 4)..)
constexpr int kGatherWarps = 8, kGatherSets = 2;         // warps 2, 3, 12..17: four for every other step
constexpr int kThreads = 32 * (2 + kEpiWarps + kGatherWarps);
constexpr int kExchBytes = 4 * 2 * 2 * 8 * 32 * 4;       // [warp pair][buffer][half][column][lane] floats
constexpr uint32_t kTmemCols = 512;
// The tensor cores cut the sum off after each instruction instead of rounding it: an error towards zero that grows
// with the length of the sum (relative, in norm: 7e-7 over 768 elements, 8e-6 over 7168, 2.7e-4 over 2^18, twice that gated).
// So a sum is made of runs of at most kRun steps, which the epilogue adds with rounding in TMEM: columns kSumCol..,
// so that a tile of more than one run has at most 128 columns.  fp32 outputs have short runs; 16-bit outputs have runs
// of 8192 elements, whose error (9e-6, gated 1.8e-5) is below a 27th of half a step of fp16 (runs of 1024: 225 against 170 us for the gated
// case of 4096 tokens above).
// Measured with runs / without, fp32 outputs: 4096 tokens gated 265 / 181 us (error 6.9e-7 / 4.2e-6), 2048 tokens, 6 of 64
// experts of 7168 -> 1024 221 / 181 us (7.2e-7 / 7.9e-6), 64 tokens of those 156 / 154 us.
constexpr int kSumCol = 128;
template <bool UP> constexpr int kRun = UP ? 6 : 12;     // steps of 64, fp32 outputs
constexpr int kRun16 = 128;                              // 16-bit outputs

struct DenseParams {
    CUtensorMap tw0, tw1;        // W, W_up: [E][rows][cols], boxes of 64 x 64
    CUtensorMap tx[4];           // x rows in place: boxes of 64 x 16, 32, 64, 128
    CUtensorMap tg;              // x rows for the gathers: boxes of 64 x 1
    const int32_t* sorted_pairs; // NULL: rows in place
    const int32_t* offsets;      // NULL: one expert over all P rows
    int E, k, P, N, K;
    bool bf16;
    void* y;
    int y_type;
    int64_t y_stride;
    int32_t* status;
    uint64_t wait_ns;
    int run;                     // steps of 64 in a run (all of them: one run)
    int max_n;                   // columns of a tile
    int stall;                   // test setting: the first wait of the MMA warp never completes
};

using Ring = RingOf<kStages>;

struct Tile {
    int e, mb, tok0, ntok, nh;   // expert, block of M rows, first sorted position, rows, columns per CTA
};
// The order of the tiles, in shared memory.  An expert's rows are cut into even blocks of at most 256.
// Experts with several blocks (whose weights are read from memory once and then found in L2: bound by
// the tensor cores) and experts with one block (bound by memory) are spread evenly among each other, so that both are
// busy all the time; in each of the two sequences the experts with the largest blocks come first, so that
// what the pairs of CTAs are left with at the end are small tiles.  Blocks of M rows are fastest:
// the pairs that run at one time share the rows of x and walk through one expert's weights.
struct Order {
    const int* off;              // [E + 1] offsets, clamped and in order
    const int* tb0;              // [n_big + 1] blocks before the i-th expert of several blocks
    const uint16_t* expert;      // experts of several blocks, then those of one
    int n_big, n_blocks, n_mb;
    uint32_t ratio;              // 2^32 * (blocks of the first sequence) / n_blocks, rounded up (0: all of them)

    // blocks of the first sequence among the first i of all
    __device__ __forceinline__ int big_before(int i) const { return ratio ? (int)__umulhi((uint32_t)i, ratio) : min(i, tb0[n_big]); }
    __device__ __forceinline__ bool at(int t, Tile& ti) const {
        const int tb = t / n_mb;
        if (tb >= n_blocks) return false;
        const int nl = big_before(tb);
        int i, nb = 1, blk = 0;
        if (big_before(tb + 1) > nl) {
            int hi = n_big;                              // tb0[i] <= nl < tb0[hi]
            for (i = 0; hi - i > 1;) {
                const int mid = (i + hi) >> 1;
                if (tb0[mid] <= nl) i = mid; else hi = mid;
            }
            nb = tb0[i + 1] - tb0[i];
            blk = nl - tb0[i];
        } else {
            i = n_big + tb - nl;
        }
        const int e = expert[i], cnt = off[e + 1] - off[e];
        const int per = ((cnt + nb - 1) / nb + 31) & ~31;    // (nb - 1) * per < cnt, as per <= 256 < cnt / (nb - 1)
        ti.e = e;
        ti.mb = t - tb * n_mb;
        ti.tok0 = off[e] + blk * per;
        ti.ntok = min(per, cnt - blk * per);
        ti.nh = ((ti.ntok + 31) & ~31) >> 1;
        return true;
    }
};
constexpr int kBuckets = 16;     // by columns of a block, 256 first: 8 for several blocks, 8 for one
__device__ __forceinline__ int blocks_of(int cnt, int max_n) { return (cnt + max_n - 1) / max_n; }
__device__ __forceinline__ int bucket_of(int cnt, int max_n) {
    if (cnt <= 0) return kBuckets;                       // no rows, no tiles
    const int nb = blocks_of(cnt, max_n), cols = ((cnt + nb - 1) / nb + 31) >> 5;
    return (nb > 1 ? 0 : 8) + 8 - cols;
}

// An epilogue warp: warp w reads TMEM lanes 32 (w % 4).. (weight rows) and every other group of columns
// (rows of x) of each tile, and stores 32 neighbouring outputs of one row at a time.
template <bool UP, typename T>
__device__ __forceinline__ void epilogue(const DenseParams& p, const Order& order, int first, int n_pairs, int cta, uint32_t tmem, float* exch, uint64_t* accf, uint64_t* accr,
                                         volatile int* abort_flag) {
    constexpr int kRowsTile = UP ? 128 : 256;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, side = (warp - kEpiWarp0) >> 2;
    const uint32_t accr0 = in_leader(su32(accr));
    const int pairbar = 1 + side * 2 + (q & 1);          // gated: warps q and q + 2 trade columns
    int j = 0, turn = 0;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const int nk = (p.K + kStepK - 1) / kStepK;
    auto complete = [&](int b) {
        bool ok = wait_warp(&accf[b], (j >> 1) & 1, abort_flag, p.wait_ns);
        // (the two warps of a trade leave together, or one would wait for the other for ever)
        if constexpr (UP) ok = all_of(pairbar, 64, ok);
        tc_after();
        return ok;
    };
    auto release = [&](int b) {
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(accr0 + 8 * b);
    };
    Tile ti;
    for (int t = first; order.at(t, ti); t += n_pairs, ++j) {
        int b = j & 1;
        if (!complete(b)) break;
        uint32_t acc = lanes + (uint32_t)b * kMaxN;
        const bool runs = p.run < nk;
        if (runs) {
            // this warp's columns of the runs, summed where it reads them from afterwards
            constexpr int kCols = UP ? 16 : 32;
            bool ok = true;
            for (int k0 = 0;;) {
                for (int c0 = kCols * side; c0 < ti.ntok; c0 += 2 * kCols)
#pragma unroll
                    for (int h = 0; h < kCols; h += 16) {
                        uint32_t r[16], s[16];
                        tmem_ld16(acc + c0 + h, r);
                        if (k0 > 0) {
                            tmem_ld16(lanes + kSumCol + c0 + h, s);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                r[i] = __float_as_uint(__fadd_rn(__uint_as_float(s[i]), __uint_as_float(r[i])));
                        } else {
                            tmem_ld_wait();
                        }
                        tmem_st16(lanes + kSumCol + c0 + h, r);
                    }
                tmem_st_wait();
                release(b);
                if ((k0 += p.run) >= nk) break;
                b = ++j & 1;
                ok = complete(b);
                if (!ok) break;
                acc = lanes + (uint32_t)b * kMaxN;
            }
            if (!ok) break;
            acc = lanes + kSumCol;
        }
        if constexpr (UP) {
            const int row = ti.mb * kRowsTile + cta * 64 + (q & 1) * 32 + lane;
            const bool is_up = q >= 2;
            // Of 16 columns the W warp keeps 0..7 and gives 8..15, the W_up warp the other way round.  The next
            // 16 are read and given before these are computed, so that their latencies overlap.
            float* const buf = exch + (pairbar - 1) * 1024 + lane;
            T* y = static_cast<T*>(p.y) + (int64_t)(ti.tok0 + 16 * side + (is_up ? 8 : 0)) * p.y_stride + row;
            float keep[8], next[8];
            auto give = [&](const uint32_t (&r)[16], float (&kept)[8]) {
                float* mine = buf + (turn & 1) * 512 + (is_up ? 256 : 0);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mine[i * 32] = __uint_as_float(is_up ? r[i] : r[8 + i]);
                    kept[i] = __uint_as_float(is_up ? r[8 + i] : r[i]);
                }
                ++turn;
            };
            uint32_t r[16];
            if (16 * side < ti.ntok) {
                tmem_ld16(acc + 16 * side, r);
                tmem_ld_wait();
                give(r, keep);
            }
            for (int c0 = 16 * side; c0 < ti.ntok; c0 += 32, y += 32 * p.y_stride) {
                const bool more = c0 + 32 < ti.ntok;
                if (more) tmem_ld16(acc + c0 + 32, r);
                named_sync(pairbar, 64);
                const float* theirs = buf + ((turn - 1) & 1) * 512 + (is_up ? 0 : 256);
                float other[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = theirs[i * 32];
                if (more) {
                    // (the other buffer: its last reader has passed the barrier above)
                    tmem_ld_wait();
                    give(r, next);
                }
                const int n = row < p.N ? ti.ntok - c0 - (is_up ? 8 : 0) : 0;
                T* at = y;
#pragma unroll
                for (int i = 0; i < 8; ++i, at += p.y_stride) {
                    const float gv = is_up ? other[i] : keep[i], uv = is_up ? keep[i] : other[i];
                    if (i < n) *at = to_out<T>(silu_times<sizeof(T) == 2>(gv, uv));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) keep[i] = next[i];
            }
        } else {
            const int row = ti.mb * kRowsTile + cta * 128 + q * 32 + lane;
            T* y = static_cast<T*>(p.y) + (int64_t)(ti.tok0 + 32 * side) * p.y_stride + row;
            for (int c0 = 32 * side; c0 < ti.ntok; c0 += 64, y += 64 * p.y_stride) {
                uint32_t r[32];
                tmem_ld32(acc + c0, r);
                tmem_ld_wait();
                const int n = row < p.N ? ti.ntok - c0 : 0;
                T* at = y;
                if (n >= 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i, at += p.y_stride) *at = to_out<T>(__uint_as_float(r[i]));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i, at += p.y_stride)
                        if (i < n) *at = to_out<T>(__uint_as_float(r[i]));
                }
            }
        }
        if (!runs) release(b);
    }
}

template <bool UP, bool IN_OUT>
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
    int* done = reinterpret_cast<int*>(tmem_slot + 2);   // [9] last step + 1 that warp 0 / each gathering warp has arrived for
    int* scan = reinterpret_cast<int*>(tmem_slot + 12);  // [20]
    int* totals = scan + 20;                             // [2] experts of several blocks, experts with rows
    int* off = totals + 2;                               // [E + 1]
    int* tb0 = off + p.E + 1;                            // [E + 1]
    uint16_t* expert = reinterpret_cast<uint16_t*>(tb0 + p.E + 1);   // [E]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t cta = cta_rank();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], p.sorted_pairs ? 2 + 2 * kGatherWarps / kGatherSets : 2); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&accf[i], 1); mbar_init(&accr[i], 2 * kEpiWarps); }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        for (int i = 0; i <= kGatherWarps; ++i) done[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tw0);
        if (UP) prefetch_map(&p.tw1);
        if (p.sorted_pairs) prefetch_map(&p.tg);
        else
            for (int i = 0; i < 4; ++i) prefetch_map(&p.tx[i]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    cluster_arrive();                                    // (barriers and TMEM are ready; waited for below)
    wait_for_previous();
    allow_next();
    // ---- the order of the tiles, from the offsets (clamped into 0..P and into order)
    bool bad = false;
    for (int i = tid; i <= p.E; i += kThreads) {
        const int o = p.offsets ? __ldg(p.offsets + i) : (i ? p.P : 0);
        bad |= o < 0 || o > p.P || (i > 0 && p.offsets && __ldg(p.offsets + i - 1) > o);
        off[i] = min(max(o, 0), p.P);
    }
    bool big = false;
    __syncthreads();
    for (int i = tid; i < p.E; i += kThreads) big |= off[i + 1] - off[i] > p.max_n;
    big = __syncthreads_or(big);
    int* hist = reinterpret_cast<int*>(exch);            // (before its use by the epilogue)
    const int n_chunks = (p.E + 31) / 32;
    if (!big) {
        // one block an expert at most: those with rows, as they come (the sort below takes 1.5 us more, and
        // only pays where many tiles of different cost follow one another)
        for (int c = warp; c < n_chunks; c += kThreads / 32) {
            const int e = 32 * c + lane;
            const unsigned m = __ballot_sync(0xffffffffu, e < p.E && off[e + 1] > off[e]);
            if (lane == 0) hist[c] = __popc(m);
        }
        __syncthreads();
        int inc = lane < n_chunks ? hist[lane] : 0;
        const int own = inc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        for (int c = warp; c < n_chunks; c += kThreads / 32) {
            const int e = 32 * c + lane, base = __shfl_sync(0xffffffffu, inc - own, c);
            const bool has = e < p.E && off[e + 1] > off[e];
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (has) expert[base + __popc(m & ((1u << lane) - 1u))] = (uint16_t)e;
        }
        if (tid == 0) { totals[0] = 0; tb0[0] = 0; }
        if (tid == 31) totals[1] = inc;
    } else {
        // experts sorted by bucket, stably (every CTA finds the same order): counts per 32 experts and
        // bucket, their running sums over the buckets, ranks
        for (int c = warp; c < n_chunks; c += kThreads / 32) {
            const int e = 32 * c + lane, k = e < p.E ? bucket_of(off[e + 1] - off[e], p.max_n) : kBuckets;
            if (lane < kBuckets) hist[c * kBuckets + lane] = 0;
            __syncwarp();
            const unsigned same = __match_any_sync(0xffffffffu, k);
            if (k < kBuckets && (same & ((1u << lane) - 1u)) == 0) hist[c * kBuckets + k] = __popc(same);
        }
        __syncthreads();
        if (warp == 0) {
            int sum = 0;
            if (lane < kBuckets)
                for (int c = 0; c < n_chunks; ++c) {
                    const int n = hist[c * kBuckets + lane];
                    hist[c * kBuckets + lane] = sum;
                    sum += n;
                }
            int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 7) totals[0] = inc;
            if (lane == 31) totals[1] = inc;
            if (lane < kBuckets) scan[lane] = inc - sum;     // first place of the bucket
        }
        __syncthreads();
        for (int c = warp; c < n_chunks; c += kThreads / 32) {
            const int e = 32 * c + lane, k = e < p.E ? bucket_of(off[e + 1] - off[e], p.max_n) : kBuckets;
            const unsigned same = __match_any_sync(0xffffffffu, k);
            if (k < kBuckets) expert[scan[k] + hist[c * kBuckets + k] + __popc(same & ((1u << lane) - 1u))] = (uint16_t)e;
        }
        __syncthreads();
        const int n_big = totals[0];
        {
            // thread t: places t * per .. of a scan of the block counts over the whole CTA
            const int per = (n_big + kThreads - 1) / kThreads, i0 = tid * per;
            auto blocks_at = [&](int i) { return blocks_of(off[expert[i] + 1] - off[expert[i]], p.max_n); };
            int sum = 0;
            for (int i = i0; i < min(i0 + per, n_big); ++i) sum += blocks_at(i);
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
            for (int i = i0; i < min(i0 + per, n_big); ++i) {
                tb0[i] = base;
                base += blocks_at(i);
            }
            if (tid == kThreads - 1) tb0[n_big] = base;
        }
    }
    tc_before();
    __syncthreads();
    cluster_wait();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int kRowsTile = UP ? 128 : 256;            // outputs of a tile of the pair
    const int n_big = totals[0];
    Order order{off, tb0, expert, n_big, tb0[n_big] + totals[1] - n_big, (p.N + kRowsTile - 1) / kRowsTile, 0u};
    if (tb0[n_big] < order.n_blocks)
        order.ratio = (uint32_t)((((uint64_t)tb0[n_big] << 32) + order.n_blocks - 1) / order.n_blocks);
    const int n_pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
    const int nk = (p.K + kStepK - 1) / kStepK;

    if (warp == 0) {
        // ======================= loads =======================
        // (the whole warp keeps step, so that what one lane issues lies in uniform registers)
        const uint32_t full0 = in_leader(su32(full)), stage0 = su32(smem);
        int g = 0;
        Ring ring;
        bool ok = true;
        Tile ti;
        for (int t = first; ok && order.at(t, ti); t += n_pairs) {
            const int c0 = uniform(ti.tok0 + (int)cta * ti.nh);  // this CTA's first column, as a sorted position
            const int r0 = uniform(ti.mb * kRowsTile + (int)cta * (kRowsTile / 2)), e = uniform(ti.e);
            // one box for the rows, of 16, 32, 64 or 128: what it reads past this block's is not used
            const int box = uniform(ti.nh > 64 ? 3 : ti.nh > 32 ? 2 : ti.nh > 16 ? 1 : 0);
            const CUtensorMap* xmap = &p.tx[box];
            const uint32_t bytes = kABytes + (p.sorted_pairs ? 0 : 2048 << box);
            for (int c = 0; c < nk * kStepK; c += kStepK, ++g, ring.next()) {
                if (!wait_warp(&empty[ring.s], ring.ph ^ 1, abort_flag, p.wait_ns)) { ok = false; break; }
                const uint32_t bar = full0 + 8 * ring.s, a = stage0 + ring.s * kStageBytes;
                if (elect_one()) {
                    arrive_tx_cluster(bar, bytes);
                    if constexpr (IN_OUT) {
                        tma_3d(a, &p.tw0, r0, c, e, bar);
                        tma_3d(a + 8192, UP ? &p.tw1 : &p.tw0, UP ? r0 : r0 + 64, c, e, bar);
                    } else {
                        tma_3d(a, &p.tw0, c, r0, e, bar);        // (128 rows at once unless gated)
                        if constexpr (UP) tma_3d(a + 8192, &p.tw1, c, r0, e, bar);
                    }
                    if (!p.sorted_pairs) tma_2d(a + kABytes, xmap, c, c0, bar);
                }
                __syncwarp();
            }
        }
        if (lane == 0) done[0] = g;
        // the last steps' arrivals on this CTA's barriers have landed before it may leave
        if (g < kStages) ring = Ring{0, 1};
        for (int i = 0; ok && i < min(g, kStages); ++i, ring.next())
            ok = wait_warp(&empty[ring.s], ring.ph ^ 1, abort_flag, p.wait_ns);
    } else if (warp == 1) {
        // ======================= MMA issue (in the first CTA) =======================
        if (cta == 0) {
            // a step's descriptors: the address field of the first stage's, plus the step's offset / 16
            const uint32_t a0 = su32(smem);
            const uint64_t da0 = IN_OUT ? sdesc_mn(a0) : sdesc(a0), db0 = sdesc(a0 + kABytes);
            constexpr uint32_t kAdvA = (IN_OUT ? 2048 : 32) >> 4, kAdvB = 32 >> 4;
            Ring ring;
            int j = 0;
            bool ok = true, any = false;
            Tile ti;
            for (int t = first; ok && order.at(t, ti); t += n_pairs) {
                const uint32_t idesc = uniform(idesc_mma(256, 2 * ti.nh, p.bf16) | (IN_OUT ? 1u << 15 : 0u));
                for (int kb = 0, start = 0, b = 0; kb < nk; ++kb, ring.next()) {
                    if (kb == start) {                               // the first step of a run
                        b = j & 1;
                        if (j >= 2 && !wait_warp(&accr[b], ((j >> 1) - 1) & 1, abort_flag, p.wait_ns)) { ok = false; break; }
                        tc_after();
                    }
                    const uint32_t acc = uniform(tmem + (uint32_t)b * kMaxN);
                    const bool first_step = kb == start, last_step = kb == nk - 1 || kb - start == p.run - 1;
                    const bool stalled = p.stall && !any;            // (test setting)
                    if (!wait_warp(stalled ? never : &full[ring.s], stalled ? 0u : ring.ph, abort_flag, p.wait_ns)) { ok = false; break; }
                    tc_after();
                    const uint32_t adv = (uint32_t)ring.s * (kStageBytes >> 4);
                    const uint64_t da = da0 + adv, db = db0 + adv;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kStepK / 16; ++kk)
                            mma_pair(acc, da + kk * kAdvA, db + kk * kAdvB, idesc, kk > 0 ? 1u : (uint32_t)!first_step);
                        commit_pair(&empty[ring.s]);
                        if (last_step) commit_pair(&accf[b]);
                    }
                    __syncwarp();
                    if (last_step) { start = kb + 1; ++j; }
                    any = true;
                }
            }
            // every MMA issued has completed before TMEM is freed
            if (any) {
                if (elect_one())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(drain))
                                 : "memory");
                __syncwarp();
                drain_wait(drain, 0, p.wait_ns);
            }
        }
    } else if (warp < kEpiWarp0 || warp >= kEpiWarp0 + kEpiWarps) {
        // ======================= gathered rows of x =======================
        if (p.sorted_pairs) {
            // warp w of a set brings rows 32 w .. of a step, four to a copy; the sets take turns (one set's
            // waits and copies took as long as a step)
            const int gw = warp < kEpiWarp0 ? warp - 2 : warp - kEpiWarps - 2, w = gw & 3, set = gw >> 2;
            const uint32_t full0 = in_leader(su32(full)), dst0 = su32(smem) + kABytes + w * 4096;
            int g = 0, last = 0;
            Ring ring;
            bool ok = true;
            Tile ti;
            int pair = 0;                                // of row 32 w + lane, read a tile ahead
            auto pair_of = [&](int t) {
                Tile n;
                const bool any = order.at(t, n);
                const int r = 32 * w + lane, c = (int)cta * n.nh + r;
                pair = any && r < n.nh && c < n.ntok ? __ldg(p.sorted_pairs + n.tok0 + c) : 0;
            };
            pair_of(first);
            for (int t = first; ok && order.at(t, ti); t += n_pairs) {
                const bool in = (uint32_t)pair < (uint32_t)p.P;
                bad |= !in;
                const int row = in ? pair / p.k : 0;
                int r[32];                               // (the same on every lane)
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __shfl_sync(0xffffffffu, row, i);
                pair_of(t + n_pairs);
                const int mine = uniform(min(max(ti.nh - 32 * w, 0), 32));   // rows: 0, 16 or 32
                for (int c = 0; c < nk * kStepK; c += kStepK, ++g, ring.next()) {
                    if ((g & 1) != set) continue;
                    if (!wait_warp(&empty[ring.s], ring.ph ^ 1, abort_flag, p.wait_ns)) { ok = false; break; }
                    const uint32_t bar = full0 + 8 * ring.s, dst = dst0 + ring.s * kStageBytes;
                    if (elect_one()) {
                        arrive_tx_cluster(bar, mine * 128);
                        if (mine >= 16) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4) tma_gather4(dst + i * 128, &p.tg, c, r[i], r[i + 1], r[i + 2], r[i + 3], bar);
                        }
                        if (mine == 32) {
#pragma unroll
                            for (int i = 16; i < 32; i += 4) tma_gather4(dst + i * 128, &p.tg, c, r[i], r[i + 1], r[i + 2], r[i + 3], bar);
                        }
                    }
                    __syncwarp();
                    last = g + 1;
                }
            }
            if (lane == 0) done[1 + gw] = last;
        }
    } else {
        // ======================= epilogue =======================
        if (p.y_type == MOE_F32) epilogue<UP, float>(p, order, first, n_pairs, (int)cta, tmem, exch, accf, accr, abort_flag);
        else if (p.y_type == MOE_BF16)
            epilogue<UP, __nv_bfloat16>(p, order, first, n_pairs, (int)cta, tmem, exch, accf, accr, abort_flag);
        else epilogue<UP, __half>(p, order, first, n_pairs, (int)cta, tmem, exch, accf, accr, abort_flag);
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
            int of[2][1 + kGatherWarps], last = 0;
            for (int i = 0; i <= kGatherWarps; ++i) {
                of[0][i] = done[i];
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(of[1][i]) : "r"(in_peer(su32(done + i))) : "memory");
                last = max(last, max(of[0][i], of[1][i]));
            }
            for (int s = max(0, last - kStages); s < last; ++s)
                for (int c = 0; c < 2; ++c) {
                    if (of[c][0] <= s) mbar_arrive(&full[s % kStages]);
                    for (int i = 1 + 4 * (s & 1); p.sorted_pairs && i <= 4 + 4 * (s & 1); ++i)
                        if (of[c][i] <= s) mbar_arrive(&full[s % kStages]);
                }
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

size_t smem_bytes(int E) {
    return 1024 + (size_t)kStages * kStageBytes + kExchBytes + (2 * kStages + 6) * 8 + 48 + 88 + 2 * (size_t)(E + 1) * 4 + 2 * (size_t)E;
}

}  // namespace

cudaError_t launch_grouped_dense(const RowsArgs& a, cudaStream_t s) {
    if (a.P <= 0) return cudaSuccess;
    DenseParams p{};
    const cuuint64_t rows = a.in_out ? a.K : a.N, cols = a.in_out ? a.N : a.K;
    const cuuint64_t wd[3] = {cols, rows, (cuuint64_t)a.E};
    const cuuint64_t ws[2] = {(cuuint64_t)a.row_stride * 2, (cuuint64_t)(a.E > 1 ? a.expert_stride : a.row_stride) * 2};
    const cuuint64_t xd[3] = {(cuuint64_t)a.K, (cuuint64_t)(a.sorted_pairs ? a.P / a.k : a.P), 1};
    const cuuint64_t xs[2] = {(cuuint64_t)a.x_stride * 2, 0};
    const CUtensorMapDataType type = a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!encode_map(&p.tw0, type, 3, a.w0, wd, ws, 64, a.in_out || a.w1 ? 64 : 128) ||
        (a.w1 && !encode_map(&p.tw1, type, 3, a.w1, wd, ws, 64, 64)))
        return cudaErrorInvalidValue;
    if (a.sorted_pairs) {
        if (!encode_map(&p.tg, type, 2, a.x, xd, xs, 64, 1)) return cudaErrorInvalidValue;
    } else {
        for (int i = 0; i < 4; ++i)
            if (!encode_map(&p.tx[i], type, 2, a.x, xd, xs, 64, 16 << i)) return cudaErrorInvalidValue;
    }
    p.sorted_pairs = a.sorted_pairs; p.offsets = a.offsets;
    p.E = a.E; p.k = a.k; p.P = a.P; p.N = a.N; p.K = a.K;
    p.bf16 = a.bf16;
    p.y = a.y; p.y_type = a.y_type; p.y_stride = a.y_stride; p.status = a.status;
    const WaitCfg wc = wait_cfg();
    p.wait_ns = wc.limit_ns; p.stall = wc.stall;
    const int nk = (a.K + kStepK - 1) / kStepK, longest = a.y_type != MOE_F32 ? kRun16 : a.w1 ? kRun<true> : kRun<false>;
    const int n_runs = (nk + longest - 1) / longest;
    p.run = (nk + n_runs - 1) / n_runs;
    p.max_n = n_runs > 1 ? kSumCol : kMaxN;
    const int v = (a.w1 ? 2 : 0) + (a.in_out ? 1 : 0);
    const void* fn = v == 3   ? (const void*)grouped_dense_kernel<true, true>
                     : v == 2 ? (const void*)grouped_dense_kernel<true, false>
                     : v == 1 ? (const void*)grouped_dense_kernel<false, true>
                              : (const void*)grouped_dense_kernel<false, false>;
    static std::atomic<uint64_t> ready[4];
    int sms = 0;
    cudaError_t err = prepare_kernel(fn, (int)smem_bytes(kMaxExperts), ready[v], &sms);
    if (err != cudaSuccess) return err;
    // one pair per two SMs, and no more pairs than there can be tiles
    const int64_t n_mb = (a.N + (a.w1 ? 127 : 255)) / (a.w1 ? 128 : 256);
    const int64_t most = ((int64_t)a.P / p.max_n + (a.E < a.P ? a.E : a.P)) * n_mb;
    const int pairs = (int)(most < sms / 2 ? most : sms / 2);
    void* args[] = {&p};
    return launch_early(fn, dim3(2 * (pairs > 0 ? pairs : 1)), kThreads, smem_bytes(a.E), s, args);
}

}  // namespace moe
