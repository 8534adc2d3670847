/*
 * moe_gb300.h -- C ABI of the GB300 (sm_103a) routed-expert MoE layer library.
 *
 * The layer: router logits -> softmax or sigmoid(+bias, group-limited) top-k
 * with renormalised gates -> token-to-expert permutation with per-expert
 * offsets -> per-expert SwiGLU FFN over GGUF block-quantized weights (Q4_K,
 * Q8_0) -> gate-weighted combine, plus an optional unweighted shared expert.
 *
 * Where the operation comes from.  The bloomery pages describe an MoE engine
 * whose routed experts run on the card over the stored GGUF quantization
 * ("bloomery README 0.3.1", Status table, "Quant types" row), whose prompt
 * batches run each expert over all its tokens at once ("bloomery V4.1
 * README", feature list, "Batched prompts"), whose decode step is one CUDA
 * graph ("bloomery README 0.3.1", "Why it is fast"), and whose router top-k
 * ids are compared exactly against a CPU reference ("bloomery early V4.1
 * README", "Oracle sets against ik_llama.cpp").  The pages print none of the
 * arithmetic; each call below states the definition it implements.
 *
 * Conventions for every call
 *  - Pointers marked (device) are CUDA device pointers owned by the caller;
 *    (host) pointers are read during the call only.  The library never
 *    allocates device memory and never synchronizes (except the two
 *    *_read_device_status calls): each call enqueues kernels on `stream` and
 *    returns, so every call can be captured in a CUDA graph.
 *  - Arguments are validated on the host before any launch; a rejected call
 *    launches nothing and returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED /
 *    MOE_ERR_WORKSPACE.  A failed launch returns MOE_ERR_CUDA.  The reason
 *    is readable with moe_last_error() (per host thread).
 *  - Weight, activation, output and workspace pointers must be 16-byte
 *    aligned; int32/fp32 routing arrays need 4-byte alignment.
 *  - Weight matrices are GGUF block rows: [rows][cols / block] blocks, the
 *    blocks running along the input dimension `cols`.  Q8_0: 34 bytes per 32
 *    weights (fp16 d, 32 x int8 q; w = d*q).  Q4_K: 144 bytes per 256
 *    weights (fp16 d, fp16 dmin, 12 bytes of packed 6-bit scales/mins for 8
 *    sub-blocks of 32, 128 bytes of 4-bit q; w = d*sc_j*q - dmin*m_j).
 *    MOE_Q8_0_R: the same Q8_0 values in moe_weights_prepare's row layout.
 *    For gate/up: rows = I, cols = H.  For down: rows = H, cols = I.
 *    Expert e of a stacked tensor starts at data + e * expert_stride_bytes.
 *  - Token-expert pairs: p = t*k + j for token t and its j-th chosen expert.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* bad pointer, size, alignment or mode */
    MOE_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement */
    MOE_ERR_WORKSPACE = 3,     /* workspace missing or smaller than the size query */
    MOE_ERR_CUDA = 4,          /* a CUDA launch or runtime call failed */
    MOE_ERR_DEVICE_CHECK = 5,  /* a device-side check failed (see *_read_device_status) */
    MOE_ERR_TIMEOUT = 6        /* a bounded device-side wait ran out (see *_read_device_status) */
} moe_status;

/* MOE_Q8_0_R: Q8_0 weights after moe_weights_prepare -- per row of K weights, the int8
 * quants of its K/32 blocks (32 bytes each, in order), then their fp16 scales, padded to
 * a multiple of 16 bytes: 32*(K/32) + roundup16(2*(K/32)) bytes a row.
 * MOE_Q5_K: 176 bytes per 256 weights -- Q4_K's 16-byte header (fp16 d, fp16 dmin, 12 bytes
 * of 6-bit scales and mins), 32 bytes whose byte i holds in bit j the 16s digit of element i
 * of sub-block j, then Q4_K's 128 nibble bytes; q in [0, 31], w = d*sc_j*q - dmin*m_j.
 * MOE_Q6_K: 210 bytes per 256 weights -- 128 bytes of low nibbles, 64 bytes of 2-bit high
 * parts, 16 int8 scales (one per 16 weights), fp16 d; element 128h + 32r + l (r < 4) takes
 * the low (r < 2) or high (r >= 2) nibble of byte 64h + 32(r % 2) + l and bits 2r, 2r + 1 of
 * byte 128 + 32h + l, u = nibble + 16 * those bits, w = d * sc[element / 16] * (u - 32).
 * MOE_Q3_K: 110 bytes per 256 weights -- 32 bytes hmask, 64 bytes of 2-bit low parts, 12
 * bytes of sixteen 6-bit scales stored + 32, fp16 d; element 128h + 32r + l takes bits 2r,
 * 2r + 1 of byte 32 + 32h + l and bit 4h + r of byte l, q = low + 4 * bit - 4 in [-4, 3]; scale
 * j: low nibble of byte 96 + j (j < 8) or high nibble of byte 96 + j - 8, bits 4-5 from bits
 * 2(j / 4).. of byte 104 + j % 4; w = d * (s_j - 32) * q.
 * MOE_MXFP4: 17 bytes per 32 weights (OCP Microscaling) -- an E8M0 scale byte e, then 16 bytes
 * whose byte j holds the FP4 E2M1 element j (low nibble) and j + 16 (high nibble);
 * w = 2^(e - 127) * e2m1 (e = 255 is NaN).  cols must be a multiple of 128.
 * These are the public GGUF layouts; the pages list them among the card-expert types
 * ("bloomery README 0.3.1", Status table, "Quant types" row), and their large model keeps its
 * routed experts as Q3_K gate and up with a Q4_K down ("bloomery README 0.3.11", limits list;
 * desc.down may have another type than gate and up).  They run on the GEMV kernels at every T
 * (moe_layer_path reports MOE_PATH_GEMV). */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_Q8_0 = 2, MOE_Q4_K = 3, MOE_Q8_0_R = 4, MOE_Q5_K = 5,
               MOE_Q6_K = 6, MOE_Q3_K = 7, MOE_MXFP4 = 8,
               MOE_F16 = 9 /* a value type of the grouped, 4-bit and norm calls only */ } moe_dtype;

typedef enum { MOE_ROUTE_SOFTMAX = 0, MOE_ROUTE_SIGMOID_GROUP = 1 } moe_route_mode;

/* One quantized weight tensor, possibly a stack of experts. */
typedef struct {
    moe_dtype qtype;             /* MOE_Q8_0, MOE_Q4_K, MOE_Q8_0_R, MOE_Q5_K, MOE_Q6_K, MOE_Q3_K or MOE_MXFP4 */
    const void* data;            /* (device) 16-byte aligned */
    int64_t rows, cols;          /* per expert; cols = input dimension */
    int64_t expert_stride_bytes; /* bytes from expert e to e+1 (multiple of 16) */
} moe_qmat;

typedef struct {
    moe_route_mode mode;
    int n_experts;               /* E, 1..1024 */
    int top_k;                   /* k, 1..min(E, 32) */
    int n_groups;                /* sigmoid mode: G divides E, G <= 32 (softmax: ignored) */
    int topk_groups;             /* sigmoid mode: groups kept, 1..G */
    float routed_scale;          /* gates are multiplied by this (1.0 = none) */
    int renormalize;             /* 1: gates renormalised over the chosen k */
} moe_route_cfg;

/* ---------------------------------------------------------------- weights */

/*
 * moe_weights_prepare -- one-time repack of a stored Q8_0 tensor (n_experts stacked
 * matrices) into MOE_Q8_0_R, the layout the kernels stream with 16-byte loads: a GGUF
 * Q8_0 block is 34 bytes, so its quants never start on a 16-byte boundary.  The values
 * are unchanged (w = d*q of the same bytes); only their place moves.  The pages' large
 * model stores its shared experts in Q8_0 ("bloomery early V4.1 README", model file
 * notes; "bloomery V4.1 README", quant-mix notes); this call lets those be read at the
 * rate of the Q4_K experts.
 *   in_out (host): the tensor to repack (qtype MOE_Q8_0, data device, 16-byte aligned,
 *     rows, cols = K a multiple of 32, expert_stride_bytes >= rows * 34 * K/32 when
 *     n_experts > 1).  On success it is rewritten to describe the repacked tensor:
 *     qtype MOE_Q8_0_R, data = dst, expert_stride_bytes = rows * row bytes.  A MOE_Q4_K
 *     tensor (and a MOE_Q5_K, MOE_Q6_K, MOE_Q3_K or MOE_MXFP4 one) is used as stored: in_out is left unchanged and
 *     nothing is written.
 *   dst (device, 16-byte aligned): at least moe_weights_prepare_size() bytes, owned by
 *     the caller; it must not overlap the source.
 * One kernel on `stream`; the source may be freed once the stream has passed it.
 */
moe_status moe_weights_prepare_size(const moe_qmat* in, int n_experts, size_t* bytes);
moe_status moe_weights_prepare(moe_qmat* in_out, int n_experts, void* dst, size_t dst_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- steps */

/*
 * moe_route -- router logits and top-k gates for T tokens.
 *   logits[t,e] = sum_h x[t,h] * W_router[e,h]          (fp32 accumulate)
 *   softmax mode: the k largest logits (ties: lower id); gates = softmax over
 *     those k (renormalize=1) or softmax over all E at those ids (0).
 *   sigmoid-group mode: s = 1/(1+exp(-l)), sel = s + bias; groups of E/G
 *     consecutive experts scored by the sum of their two largest sel; keep
 *     the topk_groups best groups (ties: lower group); the k best sel inside
 *     them; gates = s_j / sum s (renormalize=1) or s_j; the bias never enters
 *     a gate.  Gates are then multiplied by routed_scale.
 * Chosen ids are written in ascending expert id per token.
 * Pages: the router's top-k ids are integer outputs that an engine must
 * reproduce exactly outside tie bands ("bloomery early V4.1 README", "Oracle
 * sets against ik_llama.cpp"; "bloomery V4.1 README", "Against ik_llama.cpp");
 * the scoring itself is not printed there and is the definition above.
 * x (device) [T][H] in x_type (MOE_F32 or MOE_BF16); W_router (device) fp32
 * [E][H]; bias (device, nullable) fp32 [E]; logits_in (device, nullable)
 * fp32 [T][E] replaces the router product; logits_out (device, nullable) fp32
 * [T][E]; topk_ids (device) int32 [T][k]; topk_w (device) fp32 [T][k].
 * T = 0 is a no-op.
 */
moe_status moe_route(const moe_route_cfg* cfg, const void* x, moe_dtype x_type, int T, int H,
                     const float* W_router, const float* bias, const float* logits_in,
                     float* logits_out, int32_t* topk_ids, float* topk_w, moe_stream_t stream);

/*
 * moe_permute -- group the P = T*k token-expert pairs by expert.
 *   offsets[e] = number of pairs with id < e (E+1 entries, offsets[E] = P);
 *   sorted_pairs lists p in ascending (expert, p) order (stable);
 *   pair_pos[sorted_pairs[i]] = i.
 * topk_ids (device) int32 [T][k], each in [0, E) (an out-of-range id sets the
 * device status word in the workspace to MOE_ERR_DEVICE_CHECK and the pair is
 * dropped); sorted_pairs, pair_pos (device) int32 [P]; offsets (device) int32
 * [E+1]; workspace (device) of moe_permute_workspace_size() bytes.
 * Pages: a prompt batch runs each expert over all of its tokens at once
 * ("bloomery V4.1 README", feature list, "Batched prompts"); this call builds
 * that per-expert work list.  Integer work: the same bits on every run.
 */
moe_status moe_permute_workspace_size(int T, int k, int E, size_t* bytes);
moe_status moe_permute(const int32_t* topk_ids, int T, int k, int E, int32_t* sorted_pairs,
                       int32_t* offsets, int32_t* pair_pos, void* workspace, size_t ws_bytes,
                       moe_stream_t stream);

/*
 * moe_permute_noalloc -- moe_permute for callers that cannot allocate device
 * memory: code running where cudaMalloc is unavailable or forbidden (inside
 * a host callback, under an allocator lock held by an embedding runtime, or
 * in a process whose device memory is fully owned by another framework), or
 * code that must not size and pass a workspace.  The bloomery pages have no
 * counterpart of this call; it is a convenience of this library.
 * Same inputs and outputs as moe_permute, no workspace: the scratch lives in
 * a fixed 262,400-byte array inside the library that every GPU which loads
 * the library keeps until the process exits.  Limit: T*k <= 65536 pairs
 * (larger sizes return MOE_ERR_INVALID_ARG); E <= 1024 as for moe_permute.
 * Every call looks up that array's address in the current context; the first
 * call in a context may load the library's device code, so make it outside
 * any stream capture.
 * Every call on a device shares the array and zeroes its header first, so
 * two calls whose kernels overlap on the GPU (different streams, no ordering)
 * race: order them on one stream or with events.  Out-of-range ids are
 * dropped (pair_pos = -1, offsets[E] < T*k); no status word is kept.
 * Allocates nothing: no cudaMalloc, no cudaFree, no allocating library call.
 */
moe_status moe_permute_noalloc(const int32_t* topk_ids, int T, int k, int E, int32_t* sorted_pairs,
                               int32_t* offsets, int32_t* pair_pos, moe_stream_t stream);

/*
 * moe_expert_counts_add -- the running routing histogram for callers of moe_permute.
 *   Pages: the engine counts its own routing and moves the experts it calls most to the fast
 *   tier between steps ("bloomery README 0.3.1", opening feature list, MoE models larger than
 *   the card; "bloomery V4.1 README", feature list, "Adaptive residency").
 * counts[e] += offsets[e+1] - offsets[e] for e < E, one launch on `stream`.
 *   offsets (device): int32 [E+1], a moe_permute / moe_permute_noalloc result (non-decreasing);
 *   counts (device): uint64 [E], owned by the caller, read and cleared by it between calls.
 *   Atomic adds: calls on several streams may share one counts array.
 * Errors: MOE_ERR_INVALID_ARG for E outside 1..1024 or a NULL array; MOE_ERR_CUDA when the
 * launch fails.  moe_layer keeps the same histogram itself (moe_layer_desc.expert_counts).
 */
moe_status moe_expert_counts_add(const int32_t* offsets, int E, unsigned long long* counts, moe_stream_t stream);

/*
 * moe_expert_ffn -- the SwiGLU experts over the grouped pairs.
 *   for sorted position i with pair p = sorted_pairs[i], token t = p / k,
 *   expert e (offsets[e] <= i < offsets[e+1]):
 *   g = Wg[e] x_t, u = Wu[e] x_t, h = g/(1+exp(-g)) * u, y_pairs[i] = Wd[e] h.
 * gate, up: rows I, cols H; down: rows H, cols I (host structs, device data).
 * x (device) [T][H]; y_pairs (device) fp32 [T*k][H], row i = sorted position
 * i.  With sorted_pairs = NULL and offsets = NULL (then E = 1, k = 1) the
 * expert runs on every token in order, as a shared expert does.
 * fp32 accumulation, fp32 h, for every T.
 * Pages: routed experts run on the card over the file's stored block
 * quantization, Q4_K among the card types ("bloomery README 0.3.1", Status
 * table, "Quant types" row), each expert over its grouped tokens ("bloomery
 * V4.1 README", feature list, "Batched prompts").  The SwiGLU form and the
 * block layouts are not printed on the pages; they are the definitions above
 * and in the conventions at the top of this file.
 */
moe_status moe_expert_ffn_workspace_size(int T, int k, int E, int H, int I, size_t* bytes);
moe_status moe_expert_ffn(const moe_qmat* gate, const moe_qmat* up, const moe_qmat* down, int E,
                          const void* x, moe_dtype x_type, int T, int H, int I,
                          const int32_t* sorted_pairs, const int32_t* offsets, int k,
                          float* y_pairs, void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * The two halves of moe_expert_ffn, for callers that keep h or time them:
 * moe_expert_gateup writes h (device, fp32 [T*k][I], row i = sorted
 * position i) = silu(Wg[e] x_t) * (Wu[e] x_t); moe_expert_down writes
 * y_pairs[i] = Wd[e] h[i].  Same arguments and rules as moe_expert_ffn;
 * each is exactly one kernel launch.
 */
moe_status moe_expert_gateup(const moe_qmat* gate, const moe_qmat* up, int E, const void* x, moe_dtype x_type,
                             int T, int H, int I, const int32_t* sorted_pairs, const int32_t* offsets, int k,
                             float* h, moe_stream_t stream);
moe_status moe_expert_down(const moe_qmat* down, int E, const float* h, int T, int H, int I,
                           const int32_t* sorted_pairs, const int32_t* offsets, int k, float* y_pairs,
                           moe_stream_t stream);

/*
 * moe_combine -- out[t,n] = sum_{j<k} topk_w[t,j] * y_pairs[pair_pos[t*k+j], n]
 *                           (+ shared_out[t,n]) (+ old out[t,n] if accumulate),
 * summed in ascending j, then the shared term, then the old value: the same
 * bits on every run.  y_pairs, shared_out (nullable), out: fp32 (device).
 * Pages: no formula for the combine is printed; its fixed summation order
 * serves the requirement that a replay equal the eager run bit for bit
 * ("bloomery early V4.1 README", "Bit gates").
 */
moe_status moe_combine(const float* y_pairs, const float* topk_w, const int32_t* pair_pos, int T,
                       int k, int H, const float* shared_out, int accumulate, float* out,
                       moe_stream_t stream);

/*
 * moe_rmsnorm_bf16 -- u[t,h] = bf16( x[t,h] / sqrt(mean_h x[t,:]^2 + eps) * gamma[h] )
 * (fp32 arithmetic, round to nearest even).  x fp32 [T][H], gamma fp32 [H],
 * u bf16 [T][H] (device).  Used between stacked layers.
 * Pages: none of the normalisation is printed; this is the plain RMSNorm
 * definition, and the bf16 rounding is the layer input's storage type.
 */
moe_status moe_rmsnorm_bf16(const float* x, const float* gamma, int T, int H, float eps, void* u,
                            moe_stream_t stream);

/* ---------------------------------------------------------------- grouped products, unquantized experts */

/*
 * moe_grouped_matmul -- the rows of each expert times that expert's bf16 or fp16 matrix.
 *   for sorted position i of expert e (offsets[e] <= i < offsets[e+1]) and its row
 *   v = x[sorted_pairs[i] / k]  (sorted_pairs NULL: v = x[i]):
 *     w_up NULL:  y[i, n] = sum_c W[e][n, c] * v[c]
 *     w_up set :  y[i, n] = g / (1 + exp(-g)) * u,  g = W[e] v, u = W_up[e] v
 *   with n < n_out, c < n_in; products exact, sums in fp32, one rounding to y_type at the end.
 * With moe_route, moe_permute and moe_combine this is an MoE layer whose experts are stored
 * unquantized: gate and up are one call (w_up set, rows gathered through sorted_pairs), down is a
 * second one (sorted_pairs NULL, y_type MOE_F32, the y_pairs of moe_combine).
 * Pages: routed experts run each over all of its tokens at once ("bloomery V4.1 README", feature
 * list, "Batched prompts"); the pages' experts are GGUF blocks, this call serves the
 * checkpoints whose experts are not.
 *
 * desc (host, read by plan_create):
 *   type: MOE_BF16 or MOE_F16, the type of W, W_up and x;  y_type: MOE_F32, MOE_BF16 or MOE_F16;
 *   order: MOE_W_OUT_IN (expert matrices [n_out][n_in]) or MOE_W_IN_OUT ([n_in][n_out]);
 *   n_experts 1..1024, n_out and n_in 1..2^20, any value;
 *   w, w_up (device, 16-byte aligned; w_up nullable): n_experts matrices of rows row_stride
 *   elements apart (a multiple of 8, at least the row's length), expert_stride elements apart
 *   (a multiple of 8, at least (rows - 1) * row_stride + the row's length; ignored for one expert).
 * The plan keeps the pointers; the weights must outlive it and may change between calls.
 *
 * Call: x (device, 16-byte aligned) rows x_stride elements apart (a multiple of 8, >= n_in), T rows
 *   with sorted_pairs, else T*k rows; offsets (device) int32 [n_experts + 1], non-decreasing within
 *   0..T*k (NULL: one expert over all T*k rows); y (device, aligned to its type) rows y_stride >= n_out elements
 *   apart.  Rows of y outside [offsets[0], offsets[n_experts]) are left as they were.  y must not
 *   overlap x: their rows may be columns of one buffer (one stride in bytes), else their spans must not meet.
 *   status (device int32, nullable, caller-owned, never cleared by the call) is
 *   raised from MOE_OK to MOE_ERR_DEVICE_CHECK when an offset leaves 0..T*k or decreases (it is
 *   clamped) or a pair leaves 0..T*k-1 (its row of y is undefined), and to MOE_ERR_TIMEOUT when a device-side wait ran out (y is
 *   undefined).  T*k <= 2^30, strides <= 2^32; T = 0 is a no-op.  Launches one kernel, allocates nothing, needs no
 *   workspace, keeps nothing between calls: two calls may overlap on the GPU, and a captured call
 *   replays with the bits of the eager one.
 * Kernels (moe_grouped_path tells which): MOE_GROUPED_ROWS streams the weights of the experts that
 *   have rows through the warps' matrix instructions; MOE_GROUPED_TENSOR tiles 256 weight rows
 *   by up to 256 of an expert's rows on tcgen05.  Both sum in fp32, in a fixed order; long sums
 *   are made of runs that are added with rounding, so that the error of the matrix instructions, which cut their sums
 *   off, does not grow with n_in: of at most 768 elements (gated: 384) with y_type MOE_F32 (about 7e-7 relative, in
 *   norm), of at most 8192 with a 16-bit y_type, whose error (9e-6, gated 1.8e-5) is below a 27th of its half step for fp16
 *   and a 200th for bf16.
 * Errors: MOE_ERR_INVALID_ARG (NULL, size, stride, alignment), MOE_ERR_UNSUPPORTED (a type),
 *   MOE_ERR_CUDA (a launch failed).
 */
typedef enum { MOE_W_OUT_IN = 0, MOE_W_IN_OUT = 1 } moe_w_order;
typedef struct {
    moe_dtype type;              /* MOE_BF16 or MOE_F16: W, W_up and x */
    moe_dtype y_type;            /* MOE_F32, MOE_BF16 or MOE_F16 */
    moe_w_order order;
    int n_experts, n_out, n_in;
    const void* w;               /* (device) */
    const void* w_up;            /* (device, nullable) */
    int64_t row_stride, expert_stride;   /* elements */
} moe_grouped_desc;
typedef struct moe_grouped_plan moe_grouped_plan;
#define MOE_GROUPED_ROWS 0
#define MOE_GROUPED_TENSOR 1
moe_status moe_grouped_plan_create(const moe_grouped_desc* desc, moe_grouped_plan** plan);
moe_status moe_grouped_plan_destroy(moe_grouped_plan* plan);
moe_status moe_grouped_path(const moe_grouped_plan* plan, int T, int k, int* path);
moe_status moe_grouped_matmul(const moe_grouped_plan* plan, const void* x, int64_t x_stride, int T, int k,
                              const int32_t* sorted_pairs, const int32_t* offsets, void* y, int64_t y_stride,
                              int32_t* status, moe_stream_t stream);

/* ---------------------------------------------------------------- 4-bit weights with group scales */

/*
 * moe_w4_matmul -- moe_grouped_matmul over 4-bit weights with one scale per group of weights:
 *     W[e][n, c] = scale[e][n, c / group] * (q[e][n, c] - zero[e][n, c / group])
 *   q: 4-bit codes 0..15, two to a byte (weight 2j in the low nibble of byte j, 2j+1 in the high),
 *   rows dense: [n_experts][n_out][n_in / 2] bytes;  scales: fp16 or bf16 [n_experts][n_out][n_in / group];
 *   zeros (nullable): uint8 [n_experts][n_out][n_in / group], values 0..15 (the low four bits are used);
 *   NULL: every zero point is 8.  group: 32, 64 or 128;  n_in a multiple of group,
 *   at most 32768.
 * Products of q - zero and x are exact and summed in fp32 over a group, the scale is applied to that sum in fp32: no
 * weight is rounded, and one that equals its zero point adds nothing.  x is held as fp16: fp16 rows exactly, bf16 rows
 * scaled by a power of two of their largest finite magnitude, exactly down to 2^-31 of that.
 * For a few rows an expert (decode): an active expert's codes are read once for as many of its rows as are held at a time, at
 * most 16 and what fits beside the copies in flight: 16 up to n_in of about 2800, 8 up to 6400 (groups of 128: 3300 and
 * 7100), 3 or 4 at 14336, one at 32768.  More rows read them again: 2048 -> 768 gated, 8 of 128 experts, T = 16, 64, 512, 4096
 * take 61, 97, 307 and 1970 us; one expert of 14336 -> 2048 in groups of 32, T = 1, 6, 16, 64: 54, 104, 277 and 990 us.
 * Arguments, routing, y and status as moe_grouped_matmul; x of x_type MOE_BF16 or MOE_F16.
 * q, q_up 16-byte aligned; scales and zeros aligned to their element.  One launch, no workspace.
 * Pages: the card experts are 4-bit block types ("bloomery README 0.3.1", Status table, "Quant types"
 * row) in GGUF super-blocks; this is the flat form, one scale (and zero point) a group.
 */
typedef struct {
    moe_dtype x_type;            /* MOE_BF16 or MOE_F16 */
    moe_dtype y_type;            /* MOE_F32, MOE_BF16 or MOE_F16 */
    moe_dtype scale_type;        /* MOE_F16 or MOE_BF16 */
    int group;                   /* 32, 64 or 128 */
    int n_experts, n_out, n_in;
    const void* q;               /* (device) */
    const void* scales;          /* (device) */
    const uint8_t* zeros;        /* (device, nullable) */
    const void* q_up;            /* (device, nullable): the gated pair, as moe_grouped_desc.w_up */
    const void* scales_up;       /* (device) set iff q_up is */
    const uint8_t* zeros_up;     /* (device) set iff q_up and zeros are */
} moe_w4_desc;
typedef struct moe_w4_plan moe_w4_plan;
moe_status moe_w4_plan_create(const moe_w4_desc* desc, moe_w4_plan** plan);
moe_status moe_w4_plan_destroy(moe_w4_plan* plan);
moe_status moe_w4_matmul(const moe_w4_plan* plan, const void* x, int64_t x_stride, int T, int k,
                         const int32_t* sorted_pairs, const int32_t* offsets, void* y, int64_t y_stride,
                         int32_t* status, moe_stream_t stream);

/* ---------------------------------------------------------------- norms around a block */

/*
 * moe_norm_residual -- what stands between two blocks of a stack, in one pass over the rows:
 *     n = gamma_post set ? y / sqrt(mean_h y^2 + eps) * gamma_post : y     (the norm behind the block)
 *     r = res_scale * x + scale * gate * n                                 (its gate and residual scale)
 *     x_out = r                                                            (the new residual stream)
 *     u = r / sqrt(mean_h r^2 + eps) * gamma_pre                           (the norm before the next block)
 *   y: the block's output (moe_combine's out, say); all arithmetic fp32, u computed from the
 *   unrounded r, one rounding to each output's type.
 * desc (host, read during the call): H 1..32768; x_type (x and x_out), y_type, u_type: MOE_F32,
 *   MOE_BF16 or MOE_F16; gamma_post, gamma_pre (device fp32 [H], nullable); eps >= 0.
 * gate (device fp32, nullable): element (t, h) at gate[t * gate_row + h * gate_col]; (0, 1) is one
 *   gate per channel, (1, 0) one per token, (stride, 1) one per token and channel.
 * x (nullable: taken as 0), y, x_out (nullable; may be x itself, with the same stride), u (nullable;
 *   needs gamma_pre) (device): T rows, strides in elements, at least H.  x_out and u must not
 *   overlap y, each other or the gate, u must not overlap x (columns of one buffer, as for moe_grouped_matmul, do not).  Any H, stride and element-aligned pointer is accepted; rows that start on 16-byte
 *   boundaries with H a multiple of 8 are read 16 bytes at a time.
 * One launch, no workspace; T = 0 is a no-op.  Pages: none of the normalisation is printed; these
 * are the plain definitions.
 */
typedef struct {
    int H;
    moe_dtype x_type, y_type, u_type;
    const float* gamma_post;     /* (device, nullable) */
    const float* gamma_pre;      /* (device, nullable) */
    float eps, res_scale, scale;
} moe_norm_desc;
moe_status moe_norm_residual(const moe_norm_desc* desc, const void* x, int64_t x_stride, const void* y,
                             int64_t y_stride, const float* gate, int64_t gate_row, int64_t gate_col, int T,
                             void* x_out, int64_t x_out_stride, void* u, int64_t u_stride, moe_stream_t stream);

/* ---------------------------------------------------------------- dense product with its epilogue */

/*
 * moe_linear -- a dense projection and what follows it, in one kernel:
 *     y[t, n] = res_scale * r[t, n] + scale * act(sum_c W[n, c] * x[t, c] + bias[n])
 *   act: MOE_ACT_NONE; RELU max(z, 0) (NaN stays); GELU z * Phi(z), Phi the normal distribution function;
 *   GELU_TANH z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3))); SILU z / (1 + exp(-z)).
 *   Products exact, sums in fp32 in a fixed order, one rounding to y_type at the end; the activation of a 16-bit output is within
 *   2e-5 of its value, of an fp32 one within 2^-20; the tanh form of an fp32 z < 0 within 2^-20 + 5.1 w 2^-24, w = 2 sqrt(2 / pi)
 *   |z + 0.044715 z^3| its exponent, a rounded number (2^-15 where the value is not subnormal).  Long sums are made of runs of at
 *   most 768 elements with y_type MOE_F32 and 8192 with a 16-bit one, added with rounding, as those of moe_grouped_matmul; within
 *   a run the matrix instructions cut their sums off instead of rounding them (one row of 2048 elements, fp32 output: off by
 *   3.4e-7 in norm where a sum with rounding is by 7e-8; 4096 rows of 7168: 5.3e-7 and 6.4e-7).
 * The projections in front of and behind the routed experts, and dense blocks: an up half with its activation, a down
 * half that adds to the residual stream (r the stream; y may be r itself).
 * desc (host, read by plan_create):
 *   type: MOE_BF16 or MOE_F16, of W and x;  y_type, bias_type: MOE_F32, MOE_BF16 or MOE_F16;  order, n_out, n_in, w and
 *   row_stride as moe_grouped_desc for one expert;  bias (device, nullable, aligned to its type): [n_out], dense;
 *   scale, res_scale: finite.
 * The plan keeps the pointers; weights and bias must outlive it and may change between calls.
 * Call: x (device, 16-byte aligned) T rows x_stride elements apart (a multiple of 8, >= n_in); r (device, nullable) T rows of
 *   r_type, r_stride >= n_out elements apart; y (device) T rows, y_stride >= n_out; r and y aligned to their types.
 *   y may be r with r's type and stride; otherwise y must not overlap r, and never x, w or bias (columns of one
 *   buffer, as for moe_grouped_matmul, do not).  status (device int32, nullable, never cleared by the call): raised from MOE_OK to
 *   MOE_ERR_TIMEOUT when a device-side wait ran out (y is undefined).  T <= 2^30, strides <= 2^32; T = 0 is a no-op.
 *   One launch, no workspace, nothing kept between calls; a captured call replays with the bits of the eager one.
 * Kernels (moe_linear_path): MOE_LINEAR_SPLIT, tiles of 128 outputs by up to 64 rows, the sum of a tile split over a
 *   cluster of up to 8 SMs where there are few tiles; MOE_LINEAR_PAIRS, tiles of 256 outputs by up to 256 rows on pairs of SMs.
 * Errors: as moe_grouped_matmul.  Pages: the parts around the experts are not printed; these are the plain definitions.
 */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_GELU = 2, MOE_ACT_GELU_TANH = 3, MOE_ACT_SILU = 4 } moe_act;
typedef struct {
    moe_dtype type;              /* MOE_BF16 or MOE_F16: W and x */
    moe_dtype y_type;            /* MOE_F32, MOE_BF16 or MOE_F16 */
    moe_w_order order;
    int n_out, n_in;
    const void* w;               /* (device) */
    int64_t row_stride;          /* elements */
    const void* bias;            /* (device, nullable) */
    moe_dtype bias_type;
    moe_act act;
    float scale, res_scale;
} moe_linear_desc;
typedef struct moe_linear_plan moe_linear_plan;
#define MOE_LINEAR_SPLIT 0
#define MOE_LINEAR_PAIRS 1
moe_status moe_linear_plan_create(const moe_linear_desc* desc, moe_linear_plan** plan);
moe_status moe_linear_plan_destroy(moe_linear_plan* plan);
moe_status moe_linear_path(const moe_linear_plan* plan, int T, int* path);
moe_status moe_linear(const moe_linear_plan* plan, const void* x, int64_t x_stride, int T, const void* r, moe_dtype r_type,
                      int64_t r_stride, void* y, int64_t y_stride, int32_t* status, moe_stream_t stream);

/* ---------------------------------------------------------------- layer norm */

/*
 * moe_layer_norm -- per row of x, with m = mean_h x, v = mean_h (x - m)^2, q = 1 / sqrt(v + eps):
 *     y = (x - m) * q * gamma + beta;  mean[t] = m, rstd[t] = q
 * moe_layer_norm_backward -- its gradient; with xh = (x - m) * q, g = dy * gamma, from the forward call's mean and rstd:
 *     dx = add + q * (g - mean_h g - xh * mean_h(g * xh));  dgamma = sum_t dy * xh;  dbeta = sum_t dy
 *   add: the gradient that the residual stream brings along (x went into it as well), NULL: 0.
 * All arithmetic fp32, one rounding to each output's type; a row far from 0 loses nothing by its mean.
 * desc (host, read during the call): H 1..32768; x_type (x, add, dx), y_type (y, dy): MOE_F32, MOE_BF16 or
 *   MOE_F16; gamma (NULL: 1), beta (NULL: 0; not read by the backward call): device fp32 [H]; eps >= 0.
 * x, y, dy, add, dx (device): T rows, strides in elements, at least H; mean, rstd: device fp32 [T] (the forward call's may be
 *   NULL, as may y; not all three).  Any H, stride and element-aligned pointer is accepted; aligned rows (H and strides
 *   multiples of 4, pointers aligned to 4 elements; with 16-bit types alone 8 of each where they allow it) are read 8 or 16
 *   bytes at a time.
 *   y must not overlap x unless it is x, with its type and stride; dx may be add, x or dy itself (same type and
 *   stride; none of the others overlaps it).  dx, dgamma, dbeta: nullable, not all.
 * dgamma, dbeta (device fp32 [H]): overwritten, or added to with accumulate = 1; the sums over the rows have one order (the
 *   bits are those of every run).  They need a workspace (device, 256-byte aligned) of moe_layer_norm_backward_workspace_size
 *   bytes, which is free again when the call is done; calls that may overlap need one each.  dx alone needs none.
 * T <= 2^30; T = 0: nothing but dgamma = dbeta = 0 (unless accumulate).  The backward call launches two kernels,
 *   one for dx alone.
 */
typedef struct {
    int H;
    moe_dtype x_type, y_type;
    const float* gamma;          /* (device, nullable) */
    const float* beta;           /* (device, nullable) */
    float eps;
} moe_layer_norm_desc;
moe_status moe_layer_norm(const moe_layer_norm_desc* desc, const void* x, int64_t x_stride, int T, void* y, int64_t y_stride,
                          float* mean, float* rstd, moe_stream_t stream);
moe_status moe_layer_norm_backward_workspace_size(int H, int T, size_t* bytes);
moe_status moe_layer_norm_backward(const moe_layer_norm_desc* desc, const void* dy, int64_t dy_stride, const void* x,
                                   int64_t x_stride, const float* mean, const float* rstd, const void* add, int64_t add_stride,
                                   int T, void* dx, int64_t dx_stride, float* dgamma, float* dbeta, int accumulate,
                                   void* workspace, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- the router's balance */

/*
 * moe_balance_loss -- the auxiliary loss that keeps a router's load even, its counts and its gradient.
 *   p_te = softmax(logits_t)_e (MOE_ROUTE_SOFTMAX) or sigmoid(logits_te) / sum_j sigmoid(logits_tj) (SIGMOID_GROUP; a
 *   selection bias only shows in the ids).  For sequence b with n_b counted tokens:
 *     counts[b][e] = pairs of its counted tokens that name e;  f_be = E * counts[b][e] / (k * n_b);  P_be = sum_t p_te / n_b
 *     loss = coef / B' * sum_b sum_e f_be * P_be        (B': sequences with a counted token; 0 without any)
 *     dlogits_te = upstream * d loss / d logits_te      (counts held constant)
 *               = upstream * coef / (B' n_b) * p_te * (f_be - sum_j f_bj p_tj)  [sigmoid: * (1 - sigmoid(logits_te))]
 *   coef for a perfectly even load.  A logit of -inf has p = 0 and no gradient (the formula's upstream * 0: NaN with an upstream that
 *   is not finite); a token of nothing else has p = 0 throughout and a gradient of 0.
 * desc (host, read during the call): mode; n_experts 1..1024, top_k 1..min(E, 32); coef finite; accumulate.
 * logits (device, fp32): T rows, stride elements apart (>= E), as moe_route's logits_out;  ids (device, int32 [T][k]):
 *   its topk_ids;  seq_offsets (device int32 [n_seqs + 1], nullable with n_seqs = 1: one sequence of all T tokens):
 *   first tokens of the sequences, non-decreasing within 0..T; empty sequences have counts of 0;  mask (device, uint8 [T],
 *   nullable): tokens with 0 do not count (their logits and ids are not read, or not used);  upstream (device fp32 [1],
 *   nullable: 1): the gradient of what the loss goes into.
 * Outputs (device, nullable, not all): loss fp32 [1];  counts int32 [n_seqs][E];  dlogits fp32, T rows dstride apart
 *   (may be logits itself, with its stride, unless accumulating): overwritten, with 0 for tokens that do not count or that
 *   no sequence has, whatever upstream is; with accumulate added to, those tokens' rows left as they were.
 * workspace (device, 256-byte aligned): moe_balance_workspace_size bytes; it is free again when the call is done, calls that
 *   may overlap need one each.  status (device int32, nullable, never cleared by the call): raised to MOE_ERR_DEVICE_CHECK when
 *   an id of a counted token leaves 0..E-1 (it is not counted) or an offset leaves 0..T or decreases (the outputs are undefined).
 * T*k <= 2^30, n_seqs 1..65535; T = 0: loss = 0, counts = 0.  All sums have one order: the same bits each time.
 * One launch for up to 64 tokens in one or two sequences whose T * n_experts is at most 16384, two for all others.
 */
typedef struct {
    moe_route_mode mode;
    int n_experts, top_k;
    float coef;
    int accumulate;              /* 1: dlogits += */
} moe_balance_desc;
moe_status moe_balance_workspace_size(int n_experts, int T, int n_seqs, size_t* bytes);
moe_status moe_balance_loss(const moe_balance_desc* desc, const float* logits, int64_t stride, const int32_t* ids, int T,
                            const int32_t* seq_offsets, int n_seqs, const uint8_t* mask, const float* upstream, float* loss,
                            int32_t* counts, float* dlogits, int64_t dstride, int32_t* status, void* workspace, size_t ws_bytes,
                            moe_stream_t stream);

/* ---------------------------------------------------------------- fused layer */

typedef struct {
    moe_route_cfg route;
    int hidden;                   /* H */
    int intermediate;             /* I of a routed expert */
    moe_dtype x_type;             /* MOE_F32 or MOE_BF16 */
    const float* W_router;        /* (device) fp32 [E][H] */
    const float* bias;            /* (device, nullable) fp32 [E] */
    moe_qmat gate, up, down;      /* routed experts, stacked over E */
    int shared_intermediate;      /* I_s, 0 = no shared expert */
    moe_qmat s_gate, s_up, s_down;/* shared expert (single matrices) */
    int accumulate;               /* 1: out += layer(x) (a residual add); 0: out = layer(x) */
    int tc_min_tokens;            /* T at or above this uses the tensor-core path (0 = default 65) */
    int decode_chain_off;         /* 1: never use the chained decode kernels (T <= 8) */
    /* Pre-norm (nullable): x is the fp32 residual stream [T][H] (x_type MOE_F32) and the layer's
     * input is u = bf16(x / sqrt(mean_h x^2 + norm_eps) * norm_gamma), exactly as moe_rmsnorm_bf16
     * computes it; the chained decode kernels compute u themselves (no extra launch), the other
     * paths run moe_rmsnorm_bf16 into the workspace first.  With accumulate = 1 and out == x one
     * call is a whole residual block, out += layer(norm(out)).  norm_gamma: (device) fp32 [H]. */
    const float* norm_gamma;
    float norm_eps;
    /* Routing histogram (nullable): (device) uint64 [E], owned by the caller.  Every moe_layer
     * call adds, for each expert, the number of its T*k pairs routed to that expert, inside
     * the kernels that already order the pairs (no extra launch); the caller reads or clears it
     * between calls.  The pages' engine counts its own routing and moves the experts it calls
     * most to the fast tier ("bloomery README 0.3.1", opening feature list, MoE models larger
     * than the card; "bloomery V4.1 README", feature list, "Adaptive residency"). */
    unsigned long long* expert_counts;
} moe_layer_desc;

typedef struct moe_layer_plan moe_layer_plan;

/* Validates the description once and keeps a host copy of it.  Plans, workspace
 * sizes and path choice are host-side only, so the per-step launches can be
 * recorded once and replayed ("bloomery README 0.3.11", list of why it is fast:
 * one CUDA graph a decode step). */
moe_status moe_layer_plan_create(const moe_layer_desc* desc, moe_layer_plan** plan);
moe_status moe_layer_plan_destroy(moe_layer_plan* plan);
/* Bytes of device workspace moe_layer needs for up to T tokens. */
moe_status moe_layer_workspace_size(const moe_layer_plan* plan, int T, size_t* bytes);
/* Which kernels moe_layer runs for T tokens with this plan (T >= 1):
 *   MOE_PATH_GEMV         route, permute, dequant-GEMV experts and combine as
 *                         separate launches (fp32 accumulation);
 *   MOE_PATH_DECODE_CHAIN the whole layer as three launches chained by
 *                         programmatic dependent launch (router logits; routing
 *                         + gate/up; down + combine), fp32 accumulation;
 *   MOE_PATH_TENSOR       route and permute, then the tcgen05 grouped GEMM
 *                         (fp16 operands, fp32 accumulation) and combine.
 * Host-only; reads nothing on the device. */
#define MOE_PATH_GEMV 0
#define MOE_PATH_DECODE_CHAIN 1
#define MOE_PATH_TENSOR 2
moe_status moe_layer_path(const moe_layer_plan* plan, int T, int* path);
/*
 * moe_layer -- the whole layer: route, permute, experts, combine (+ shared),
 * for T tokens of x (device, [T][H] in desc->x_type) into out (device, fp32
 * [T][H]).  Enqueued on `stream` with no host synchronization and no host
 * read-back, so it can be captured in a CUDA graph; replays give the same
 * bits as eager calls.  The expert path is chosen from T on the host
 * (moe_layer_path tells which): T <= 8 (T*k <= 64, E <= 256, Q4_K routed
 * experts, H <= 2048, the staged x and the gate/up rings within the kernel's
 * shared memory: T <= 6 at H = 2048) the chained decode kernels, T < tc_min_tokens the fp32
 * dequant-GEMV kernels (both fp32 accumulate), larger T the tensor-core
 * grouped GEMM (fp16 operands, fp32 accumulate; the per-pair down outputs
 * are rounded to fp16 before the fp32 combine).  out may alias x when
 * accumulate = 1 (a residual block): x is read before out is written.
 * T = 0 is a no-op that launches nothing (x, out and workspace may be NULL).
 * Pages: one CUDA graph per decode step ("bloomery README 0.3.11", list of why
 * it is fast), prompts as tensor-core GEMMs (same list) over experts grouped by
 * token ("bloomery V4.1 README", feature list, "Batched prompts"), and a graph
 * replay that equals the eager run bit for bit ("bloomery early V4.1 README",
 * "Bit gates").
 */
moe_status moe_layer(const moe_layer_plan* plan, const void* x, int T, float* out, void* workspace,
                     size_t ws_bytes, moe_stream_t stream);
/* moe_layer that also records two caller-owned CUDA events (cudaEvent_t, may
 * be NULL) on `stream` immediately before and after the launch of the routed
 * gate/up kernel, so a caller can time that kernel alone.  Same results as
 * moe_layer; meant for eager calls (not for graph capture). */
moe_status moe_layer_timed(const moe_layer_plan* plan, const void* x, int T, float* out, void* workspace,
                           size_t ws_bytes, moe_stream_t stream, void* ev_before_gateup, void* ev_after_gateup);

/* Device pointers into a moe_layer workspace (any output may be NULL) to
 * the last call's ids int32 [T][k], gates fp32 [T][k] and offsets int32
 * [E+1]. */
moe_status moe_layer_debug_views(const moe_layer_plan* plan, int T, void* workspace,
                                 int32_t** topk_ids, float** topk_w, int32_t** offsets);

/* Copies the device status word of a workspace (MOE_OK or a MOE_ERR_* code
 * raised by a device-side check) to *code and clears it.  Synchronizes the
 * stream first; call it outside graph capture.  Pages: a bad request is
 * refused by name rather than run ("bloomery README 0.3.11", limits list). */
moe_status moe_read_device_status(const moe_layer_plan* plan, int T, void* workspace, int32_t* code,
                                  moe_stream_t stream);
moe_status moe_permute_read_device_status(int T, int k, int E, void* workspace, int32_t* code,
                                          moe_stream_t stream);

/*
 * moe_debug_set_waits -- test hook for the bounded device-side waits; off by
 * default.  Every wait of the library's kernels on a copy or an MMA gives up
 * after limit_ns nanoseconds (0 restores the default of 2 s), records
 * MOE_ERR_TIMEOUT in the workspace status word (the call's status argument for the grouped,
 * 4-bit and dense products), waits (within the same limit)
 * for the copies its CTA still has in flight, releases what it holds and
 * returns; the call's outputs are then undefined and moe_read_device_status
 * reports the code.  stall = 1 makes the first wait of the chained decode,
 * segmented GEMV, tensor-core, grouped, 4-bit and dense-product kernels wait on a barrier that nothing
 * completes, so that a test can run this path without a faulty input.
 * Applies to calls launched after it, from any host thread (a graph keeps the
 * setting it was captured with).  The failure reporting follows the pages'
 * refusals by name with named exit codes ("bloomery README 0.3.11").
 */
moe_status moe_debug_set_waits(uint64_t limit_ns, int stall);

/*
 * moe_debug_set_stamps -- timing hook of the chained decode kernels (T <= 8); off by
 * default (buf = NULL).  With a device buffer of at least 3*256*8*8 = 49,152 bytes, every
 * chained call launched afterwards has thread 0 of CTA c (c < 256) of kernel n (0 router
 * logits, 1 routing + gate/up, 2 down + combine) write the GPU's global nanosecond clock
 * at phase ph into buf[(n*256 + c)*8 + ph] (uint64): n = 0: 0 start, 1 after the wait for
 * the previous launch, 2 router dot products done, 3 end; n = 1: 0 start, 1 activations
 * staged, 2 after the wait, 3 routing read, 4 first unit computed, 5 units done, 6 CTA
 * done, 7 top-k written; n = 2: 0 start, 2 routing read and down rows requested (before
 * the wait), 1 after the wait, 3 h copies issued, 4 copies landed, 5 dot products done, 6 CTA
 * done.  Calls overwrite the same slots; a graph keeps the setting it was
 * captured with.  For measuring where a decode layer's time goes; the results are
 * unchanged.  Pages: step times there are quoted with their instrumentation state
 * ("bloomery early V4.1 README", caveats of the depth measurement).
 */
moe_status moe_debug_set_stamps(void* buf, size_t bytes);

/* The reason for the last non-MOE_OK status returned on this host thread
 * (refusals by name: "bloomery README 0.3.11", limits list). */
const char* moe_last_error(void);
/* Library version string. */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
