/*
 * gmm.h — C ABI of the GB300 (sm_103a) ragged grouped GEMM library (libgmm.so).
 *
 * The operation (Modular "grouped_matmul_sm100_persistent" API page, section
 * "Args"): for every group g whose expert id e = expert_ids[g] satisfies
 * 0 <= e < num_experts,
 *
 *     C[r, n] = bf16( sum_k A[r, k] * B[e, n, k] )
 *         for r in [a_offsets[g], a_offsets[g+1]), n in [0, N)
 *
 * accumulated in fp32 on the tensor cores and rounded to nearest even.
 *   - A  : bf16 [rows, K], row-major (K contiguous).  rows >= a_offsets[num_groups].
 *   - B  : bf16 [num_experts, N, K], row-major — the transposed-B convention of the
 *          page (each expert's weight matrix is stored N x K).
 *   - C  : bf16 [rows, N], row-major.
 *   - a_offsets          : uint32 [num_groups + 1], non-decreasing prefix sum of rows per group.
 *   - expert_ids         : int32  [num_groups]; a negative id skips the group.
 *   - expert_usage_stats : uint32 [>= 2]; index 1 receives the number of groups with
 *                          0 <= id < num_experts.  No other entry is read or written.
 * Rows of C that no active group covers keep their previous contents, bit for bit.
 *
 * Device-side conventions (checked on the device, reported by gmm_query_status):
 *   - a decreasing a_offsets entry: nothing is computed, stats[1] is still written,
 *     status GMM_ERR_BAD_INPUT;
 *   - an expert id >= num_experts: that group is skipped and not counted,
 *     status GMM_ERR_BAD_INPUT.
 *
 * All pointers passed to the run calls are DEVICE pointers on the handle's device
 * and are owned by the caller.  The run calls are asynchronous on `stream`: they
 * validate the arguments on the host, launch one persistent kernel and return;
 * they do not synchronise and allocate nothing.  They can be captured in a CUDA
 * graph and replayed (every device write they make before the kernel is a value
 * write, not a copy from host memory); gmm_query_status synchronises and must not
 * be called during a capture.
 *
 * A handle owns a small device workspace (a status word, a 64-bit tile-claim
 * word and a finished-CTA counter that each launch returns to zero, the routing of
 * gmm_matmul_int4's single group, per-CTA tensor-map slots, and the chunk counts of
 * gmm_dispatch) that every launch made through it rewrites.  Launches made through the
 * same handle must therefore not overlap on the GPU: issue them on one stream, or
 * use one handle per stream.  (gmm_route, gmm_route_grad, the gmm_quantize_fp8 calls and
 * gmm_weight_grad_fp8 use nothing of it but the status word, and may overlap with one
 * another and with other calls.)
 */
#ifndef GMM_H_
#define GMM_H_

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes.  0 is success; everything else is negative. */
#define GMM_OK                  0
#define GMM_ERR_INVALID_ARG    -1  /* null pointer, negative size, misaligned or badly shaped operand */
#define GMM_ERR_UNSUPPORTED    -2  /* valid request outside what the kernels implement (e.g. too many groups) */
#define GMM_ERR_CUDA           -3  /* a CUDA runtime/driver call failed (allocation, launch, copy) */
#define GMM_ERR_DEVICE_TIMEOUT -4  /* a kernel gave up waiting on its own pipeline (reported by gmm_query_status) */
#define GMM_ERR_BAD_INPUT      -5  /* decreasing a_offsets, or an expert id, slot or row index past its range
                                      (gmm_query_status) */
#define GMM_ERR_NO_DEVICE      -6  /* the device is not an sm_103 GPU, or none is present */

typedef struct gmm_ctx *gmm_handle_t;

/*
 * Create a handle for `device` and `num_experts` experts (E, the leading
 * dimension of B; used for the id bounds check and the B tensor map).  This is
 * the host-side set-up that the grouped GEMM page's launcher does before its
 * persistent kernel (Modular "grouped_matmul_sm100_persistent", description: it
 * builds the TMA descriptors and picks the pipeline depth from the shared memory
 * available): here every kernel's shared-memory budget is read from the device's
 * opt-in shared memory once, each launch sizes its rings beside that call's group
 * prefix, and the tensor maps are built per call.
 * Allocates the handle's device workspace on `device` (cudaMalloc).  The
 * caller's current device is left unchanged.
 * Errors: GMM_ERR_INVALID_ARG (out == NULL, num_experts < 1),
 *         GMM_ERR_NO_DEVICE (no such device, or not compute capability 10.3),
 *         GMM_ERR_CUDA (allocation failed, or a kernel's launch configuration could
 *         not be set up).  *out is NULL on error.
 */
int gmm_create(gmm_handle_t *out, int num_experts, int device);

/*
 * bf16 ragged grouped GEMM (see the header comment for the operation).
 * N and K: multiples of 8 (16-byte rows, a TMA requirement), both >= 8.
 * c, a, b: 16-byte aligned.  num_groups: 0 .. 4096.
 * With num_groups == 0 only expert_usage_stats[1] = 0 is written (expert_ids may then be NULL).
 * A call without rows (a batch that gave this device no tokens) has c and a both NULL, as
 * an empty tensor's pointer is: all its groups are empty, a_offsets is not read, and only
 * expert_usage_stats[1] is written.  The other grouped calls of a handle take it too.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED,
 *         GMM_ERR_CUDA (tensor-map encoding or launch failed).
 */
int gmm_run(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
            const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
            cudaStream_t stream);

/*
 * Optional elementwise epilogue, applied to each fp32 result before it is rounded
 * to bf16 (the grouped and quantised GEMM pages both take an optional elementwise
 * function on the output: Modular "grouped_matmul_sm100_persistent" and
 * "multistage_gemm_q", section "Parameters", elementwise_lambda_fn; a C interface
 * takes these common steps instead of a function):
 *     y = act( acc[r, n] + bias[e, n] ) * row_scale[r]
 * where e is the group's expert and r the row of A.  Each part is optional:
 *   bias:       bf16 [num_experts, N] (2-byte aligned), or NULL for none;
 *   row_scale:  fp32 [rows of A] (4-byte aligned, e.g. routing weights), or NULL;
 *   activation: GMM_ACT_NONE, GMM_ACT_RELU (max(y, 0)), GMM_ACT_SILU (y / (1 + e^-y)),
 *               GMM_ACT_GELU_TANH (y/2 (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3)))).
 * Rows that no active group covers stay untouched, as without the epilogue.
 */
#define GMM_ACT_NONE      0
#define GMM_ACT_RELU      1
#define GMM_ACT_SILU      2
#define GMM_ACT_GELU_TANH 3

typedef struct gmm_epilogue {
  const void *bias;
  const float *row_scale;
  int activation;
} gmm_epilogue;

/*
 * gmm_run with the optional epilogue (epilogue == NULL: exactly gmm_run).
 * Errors: as gmm_run, plus GMM_ERR_INVALID_ARG for an unknown activation or a
 * misaligned bias / row_scale.
 */
int gmm_run_ex(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
               const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
               const gmm_epilogue *epilogue, cudaStream_t stream);

/*
 * 4-bit grouped GEMM (the grouped path with the weights of Modular's
 * "multistage_gemm_q", section "Parameters": pack_factor 4-bit values per uint32 and
 * one scale per group_size K elements).  B[e, n, k] is replaced by
 *     w = bf16( (q - 8) * scale[e, n, k / group_size] ),
 *     q = bits [4*(k%8), 4*(k%8)+4) of b_packed[e, n, k/8]   (low nibble first),
 * b_packed: uint32 [num_experts, N, K/8] (16-byte aligned);
 * b_scales: bf16 [num_experts, N, K/group_size] (2-byte aligned).
 * Requirements: those of gmm_run, plus group_size a multiple of 64 that divides K.
 * Errors: as gmm_run.
 */
int gmm_run_int4(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets,
                 const uint32_t *b_packed, const void *b_scales, const int32_t *expert_ids,
                 uint32_t *expert_usage_stats, int num_groups, int N, int K, int group_size,
                 cudaStream_t stream);

/*
 * Dense rank-2 4-bit GEMM (Modular "multistage_gemm_q": C = A . B^T with B packed
 * 4-bit and group-quantised, section "Parameters": pack_factor, group_size):
 *     C[r, n] = sum_k A[r, k] * w[n, k],  w[n, k] = bf16( (q - 8) * scale[n, k / group_size] )
 * for r < M, with the nibble layout of gmm_run_int4.  It is the grouped path with one
 * group of M rows and one expert; the group's offsets and id are written into the
 * handle's workspace (stream-ordered), so the caller passes none.
 *   c: bf16 [M, N]; a: bf16 [M, K]; b_packed: uint32 [N, K/8]; b_scales: bf16 [N, K/group_size].
 * The page's function raises when an operand is not rank-2; here the ranks are fixed
 * by the signature (the Python binding raises for tensors of another rank).
 * M == 0 launches nothing.  Requirements and errors: as gmm_run_int4_ex, plus
 * GMM_ERR_INVALID_ARG for M < 0.  Calls through one handle share its workspace, so
 * they must be stream-ordered, as for every call through a handle.
 */
int gmm_matmul_int4(gmm_handle_t h, void *c, const void *a, const uint32_t *b_packed, const void *b_scales,
                    int M, int N, int K, int group_size, const gmm_epilogue *epilogue, cudaStream_t stream);

/* gmm_run_int4 with the optional epilogue (epilogue == NULL: exactly gmm_run_int4). */
int gmm_run_int4_ex(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets,
                    const uint32_t *b_packed, const void *b_scales, const int32_t *expert_ids,
                    uint32_t *expert_usage_stats, int num_groups, int N, int K, int group_size,
                    const gmm_epilogue *epilogue, cudaStream_t stream);

/*
 * The bf16 grouped GEMM with A-plane row offsetting (Modular
 * "grouped_matmul_sm100_persistent", section "Parameters": a_plane_splits, per-plane
 * split sizes for fused LoRA QKV A-plane row offsetting, (0, 0) disabling it).  The
 * reading taken: a holds three planes of M = a_offsets[G] rows, stacked along its rows
 * ([3 M, K], e.g. the q, k and v inputs of a fused QKV projection), and
 * (s0, s1) = a_plane_splits cut the N columns into three parts:
 *     C[r, n] = bf16( sum_k a[p(n) * M + r, k] * b[e, n, k] ),
 *     p(n) = 0 for n < s0, 1 for s0 <= n < s0 + s1, 2 otherwise,
 * for the rows and groups of gmm_run, then the optional epilogue.  (0, 0) is gmm_run_ex.
 * a must hold 3 * a_offsets[G] rows (any a_offsets[G] rows when the splits are (0, 0)).
 * Requirements: those of gmm_run, s0 and s1 multiples of 256 (a tile's 256 weight rows
 * lie in one plane; else GMM_ERR_UNSUPPORTED), 0 <= s0, 0 <= s1, s0 + s1 <= N (else
 * GMM_ERR_INVALID_ARG, also for a NULL a_plane_splits).  Errors: as gmm_run_ex.
 */
int gmm_run_planes(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                   const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                   const int *a_plane_splits, const gmm_epilogue *epilogue, cudaStream_t stream);

/*
 * Block-scaled e4m3 grouped GEMM (Modular "k_matmul_ragged_paged_scale", section
 * "Args": input_scale and weight_scale multiply the input and the weight; template
 * parameter scales_granularity_mnk; without the page's paged KV-cache write, the
 * result goes to C as in gmm_run).  With (gm, gn, gk) = scales_granularity_mnk and
 * kb = k / gk the K block of k:
 *     C[r, n] = bf16( sum_kb input_scale[r / gm, kb] * weight_scale[e, n / gn, kb]
 *                            * sum_{k in block kb} a[r, k] * b[e, n, k] )
 * for the rows and groups of gmm_run, a and b e4m3 (1 sign, 4 exponent bits with
 * bias 7, 3 mantissa bits), sums in fp32.  Then the optional epilogue.
 *   a: e4m3 bytes [rows, K] (16-byte aligned); b: e4m3 bytes [num_experts, N, K]
 *   (16-byte aligned); input_scale: fp32 [ceil(rows / gm), ceil(K / gk)] (without rows it
 *   may be NULL);
 *   weight_scale: fp32 [num_experts, ceil(N / gn), ceil(K / gk)] (both row-major,
 *   4-byte aligned, read only for active groups); c and the rest as gmm_run.
 * Requirements: those of gmm_run with K a multiple of 16 (an e4m3 row is K bytes, a
 * multiple of 16 for TMA), gm, gn, gk >= 1, and either gk >= K (one scale over the
 * whole reduction, applied to the finished sum) or gk a multiple of 128 with gn a
 * multiple of 32 (per-K-block scales, a kernel of their own); other granularities
 * return GMM_ERR_UNSUPPORTED.
 * Errors: as gmm_run_ex, plus GMM_ERR_INVALID_ARG for NULL or misaligned scales,
 * a NULL scales_granularity_mnk or a granularity below 1.
 */
int gmm_run_fp8(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                const float *input_scale, const float *weight_scale, const int *scales_granularity_mnk,
                const gmm_epilogue *epilogue, cudaStream_t stream);

/* Element types of logits, tokens and rows. */
#define GMM_DTYPE_BF16 0
#define GMM_DTYPE_FP16 1
#define GMM_DTYPE_FP32 2

/*
 * A router's choice: the experts of each token and their weights, from its logits x.
 *   score       s_e = softmax(x)_e, or 1 / (1 + exp(-x_e));
 *   key         y_e = s_e + bias[e]: what the choice goes by (bias: fp32 [num_experts] or NULL;
 *               it moves load between experts and does not enter the weights);
 *   groups      expert_groups equal runs of experts (1: none).  A group's key is the sum of its
 *               group_top (1 or 2) largest y_e; the top_groups groups with the largest keys stay;
 *   choice      the top_k largest y_e of the groups that stay, in descending order;
 *   weights     scale * s_j, or with renormalise scale * s_j / (the sum of the chosen s_j).
 * Equal keys, of experts or of groups, go to the lowest index.  Keys are compared to 64-bit
 * accuracy, single scores without a bias (which stand in the order of the logits) as the logits;
 * equal logits of equal bias are equal keys.  Scores and weights are fp32.
 * An expert whose key is -infinity or NaN (a masked logit or bias) is never chosen; a group's key
 * leaves such experts out.  A slot that finds no expert gets id -1 and weight 0, which
 * gmm_dispatch drops.  A token with a NaN logit (softmax: or one of +infinity) gets no expert and
 * is reported as GMM_ERR_BAD_INPUT by gmm_query_status.
 */
#define GMM_SCORE_SOFTMAX 0
#define GMM_SCORE_SIGMOID 1

typedef struct gmm_route_options {
  int scoring;          /* GMM_SCORE_* */
  int expert_groups;
  int top_groups;
  int group_top;
  int renormalise;      /* 0 or 1 */
  float scale;          /* finite, above zero */
} gmm_route_options;

/*
 *   slot_experts : int32 [num_tokens, top_k], written;  weights: fp32 [num_tokens, top_k], written
 *                  (gmm_dispatch's and gmm_combine's operands);
 *   logits       : [num_tokens, num_experts] of `dtype`, num_experts the handle's, rows
 *                  logits_stride elements apart (0: one row for all).
 * num_tokens == 0 launches nothing.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG (NULL or misaligned for its element type,
 * negative size, unknown dtype or option, expert_groups that does not divide num_experts,
 * top_groups above expert_groups, group_top above a group's experts, top_k above the experts
 * that can stay), GMM_ERR_UNSUPPORTED (top_k > 32, more than 2^30 slots, more than 4096 experts,
 * 32 groups, or 128 experts a group and lane: a group has 32 / expert_groups lanes, rounded down
 * to a power of two), GMM_ERR_CUDA.
 */
int gmm_route(gmm_handle_t h, int32_t *slot_experts, float *weights, const void *logits, long long logits_stride,
              const float *bias, int num_tokens, int top_k, int dtype, const gmm_route_options *options,
              cudaStream_t stream);

/*
 * The gradient of the weights for the logits, the choice held fixed: d_logits = sum over a token's
 * slots of d_weights * d weight / d logit, zero for logits that do not enter (fp32, rounded once).
 *   d_logits     : [num_tokens, num_experts] of `dtype`, rows d_logits_stride (>= num_experts)
 *                  elements apart, written whole;
 *   d_weights    : fp32 [num_tokens, top_k]; a slot with a negative id or a logit of -infinity is
 *                  left out, an id >= num_experts too and is reported as GMM_ERR_BAD_INPUT; slots
 *                  of a token that name an expert twice both count;
 *   slot_experts, logits: as gmm_route wrote and took them; options: its scoring, renormalise and
 *   scale (the others are not read).  A token that gmm_route reports gets zeros.
 * Errors: as gmm_route.
 */
int gmm_route_grad(gmm_handle_t h, void *d_logits, long long d_logits_stride, const float *d_weights,
                   const int32_t *slot_experts, const void *logits, long long logits_stride, int num_tokens, int top_k,
                   int dtype, const gmm_route_options *options, cudaStream_t stream);

/*
 * Tokens sorted by expert and back.  A router gives token t its top_k experts; slot
 * s = t * top_k + j is its j-th.  Rows (the grouped calls' A and C) hold one slot each, all
 * slots of expert 0 first, then expert 1, ..., each expert's in ascending slot order.
 * The calls below are asynchronous on `stream`, allocate nothing, can be captured in a CUDA
 * graph, and give the same bits every time (gmm_combine_grad for distinct rows, which it
 * requires).
 */

/*
 * Sort the slots by expert and copy the tokens to their rows.
 *   slot_experts : int32 [num_tokens, top_k]; a negative id drops the slot, an id
 *                  >= num_experts (the handle's) drops it and is reported as
 *                  GMM_ERR_BAD_INPUT by gmm_query_status.  A token may name an expert twice.
 *   a_offsets    : uint32 [num_experts + 1], written: the prefix sum of rows per expert, for
 *                  grouped calls with num_groups = num_experts and expert_ids = 0, 1, ....
 *   slot_rows    : int32 [num_tokens, top_k], written: each slot's row, -1 for a dropped one.
 *   row_slots    : int32 [num_tokens * top_k], written: each row's slot, -1 for the rows at
 *                  and past a_offsets[num_experts].
 *   rows         : [num_tokens * top_k, width], contiguous, written below
 *                  a_offsets[num_experts]: rows[r, :] = tokens[row_slots[r] / top_k, :].
 *   tokens       : [num_tokens, width] of `dtype`, rows tokens_stride elements apart (0: one
 *                  row for all).  rows and tokens both NULL: only the sort.
 * The gradient of the copy, d_tokens[t, :] = sum_j d_rows[slot_rows[t, j], :], is
 * gmm_combine without weights.
 * num_tokens == 0 writes a_offsets only.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG (NULL or misaligned for its element
 * type, negative size, unknown dtype, only one of rows and tokens), GMM_ERR_UNSUPPORTED
 * (top_k > 32, more than 2^30 slots, width > 2^31 - 4096, more than 4096 experts), GMM_ERR_CUDA.
 */
int gmm_dispatch(gmm_handle_t h, uint32_t *a_offsets, int32_t *slot_rows, int32_t *row_slots, void *rows,
                 const int32_t *slot_experts, const void *tokens, long long tokens_stride, int num_tokens, int top_k,
                 int width, int dtype, cudaStream_t stream);

/*
 * Rows back to tokens, weighted:
 *     out[t, :] = sum_j weights[t, j] * rows[slot_rows[t, j], :]
 * summed in fp32 in ascending j and rounded once; a negative slot_rows entry adds nothing
 * (a token with none gets zeros), one >= num_rows adds nothing and is reported as
 * GMM_ERR_BAD_INPUT.
 *   out: [num_tokens, width] of `dtype`, rows out_stride (>= width) elements apart;
 *   rows: [num_rows, width], contiguous; slot_rows: int32 [num_tokens, top_k];
 *   weights: fp32 [num_tokens, top_k], or NULL for ones.
 * Errors: as gmm_dispatch (the number of experts does not matter).
 */
int gmm_combine(gmm_handle_t h, void *out, long long out_stride, const void *rows, int num_rows, const int32_t *slot_rows,
                const float *weights, int num_tokens, int top_k, int width, int dtype, cudaStream_t stream);

/*
 * The gradient of gmm_combine:
 *     d_rows[slot_rows[t, j], :] = weights[t, j] * d_out[t, :]
 *     d_weights[t, j] = sum_n d_out[t, n] * rows[slot_rows[t, j], n]     (0 for a dropped slot)
 *   d_rows: [num_rows, width], contiguous; rows that no slot names stay untouched;
 *   slot_rows: the rows that it names (those in 0 .. num_rows - 1) must be distinct, as
 *   gmm_dispatch's are, also where a token names an expert twice.  This is not checked: a
 *   row that several slots name receives their products element by element in no particular
 *   order, not the sum (gmm_combine itself may name a row more than once);
 *   d_weights: fp32 [num_tokens, top_k], or NULL (rows may then be NULL too);
 *   d_out: [num_tokens, width], rows d_out_stride elements apart (0: one row for all);
 *   rows, weights: as gmm_combine took them.
 * Products and sums in fp32 (each element of d_rows rounded once).  Errors: as gmm_combine.
 */
int gmm_combine_grad(gmm_handle_t h, void *d_rows, float *d_weights, const void *d_out, long long d_out_stride,
                     const void *rows, int num_rows, const int32_t *slot_rows, const float *weights, int num_tokens,
                     int top_k, int width, int dtype, cudaStream_t stream);

/*
 * 8-bit floating point (e4m3) with a scale for each block of 128:
 *     q = e4m3(x / s),  s = amax / 448  (amax: the block's largest magnitude)
 * every step rounded to nearest even in fp32, s = 0 giving q = 0; with pow2 = 1, s is the smallest
 * power of two that is at least amax / 448 (2^-127 at least; 0 for a block of zeros).  A block that
 * holds an infinity or a NaN gets a NaN scale and zero codes.
 *
 * Rows, a scale for each 128 elements of a row: gmm_run_fp8's a and input_scale of granularity
 * (1, ., 128), optionally gathered.
 *   q: e4m3 [rows, K] (16-byte aligned); scales: fp32 [rows, ceil(K / 128)];
 *   x: [src_rows, K] of `dtype`, rows x_stride elements apart (0: one row for all);
 *   row_slots: int32 [rows] (gmm_dispatch's row_slots) or NULL: row r is quantised from
 *   x[row_slots[r] / top_k]; a row with a negative entry stays untouched, one whose source row is
 *   past src_rows too and is reported as GMM_ERR_BAD_INPUT.
 * Requirements: K a multiple of 16, up to 2^24; rows up to 2^30.  rows == 0 launches nothing.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED, GMM_ERR_CUDA.
 */
int gmm_quantize_fp8(gmm_handle_t h, void *q, float *scales, const void *x, long long x_stride, int src_rows,
                     const int32_t *row_slots, int top_k, int rows, int K, int dtype, int pow2, cudaStream_t stream);

/*
 * Weights, a scale for each 128 x 128 of a matrix: gmm_run_fp8's b and weight_scale of granularity
 * (., 128, 128).  The codes of the transposed weights, for the product that takes gradients back
 * through the layer, are these transposed, with the scales transposed.
 *   q: e4m3 [batch, N, K] (16-byte aligned); scales: fp32 [batch, ceil(N / 128), ceil(K / 128)];
 *   x: [batch, N, K] of `dtype`, contiguous.
 * Requirements and errors: as gmm_quantize_fp8, and up to 2^31 - 1 tiles.
 */
int gmm_quantize_fp8_tiles(gmm_handle_t h, void *q, float *scales, const void *x, int batch, int N, int K, int dtype,
                           int pow2, cudaStream_t stream);

/*
 * Along the rows of each group, a scale for each 128 rows and column: the operands of
 * gmm_weight_grad_fp8.  The codes are stored transposed, and each group's rows start a block:
 *     q_t[c, at(r)] for r in [a_offsets[g], a_offsets[g+1]),
 *     at(r) = (a_offsets[g] / 128 + g) * 128 + (r - a_offsets[g])
 * with zeros behind a group's last row up to the end of its block.  Scales are powers of two, as
 * their exponent codes (2^(code - 127); 0 for a block of zeros, 255 for NaN).
 *   q_t: e4m3 [width, pitch], pitch = GMM_FP8_COLS_PITCH(rows, num_groups) (16-byte aligned);
 *   t_scales: uint8 [pitch / 128, width]; blocks that no group uses stay untouched in both;
 *   q, scales: both NULL, or written too, of the rows that a group covers, as gmm_quantize_fp8
 *   with pow2 = 0 writes them (the rows are read once for both forms);
 *   x, row_slots, top_k: as gmm_quantize_fp8; a row without a source counts as zeros in q_t;
 *   a_offsets: uint32 [num_groups + 1], non-decreasing, at most rows; else nothing is written, and
 *   GMM_ERR_BAD_INPUT is reported by gmm_query_status.
 * Requirements: width a multiple of 16, up to 2^24; num_groups up to 4096.  rows == 0 or
 * num_groups == 0 launches nothing.  Errors: as gmm_quantize_fp8, plus GMM_ERR_INVALID_ARG for only
 * one of q and scales.
 */
#define GMM_FP8_COLS_PITCH(rows, num_groups) (((rows) / 128 + (num_groups)) * 128)
int gmm_quantize_fp8_cols(gmm_handle_t h, void *q_t, void *t_scales, void *q, float *scales, const void *x,
                          long long x_stride, int src_rows, const int32_t *row_slots, int top_k, const uint32_t *a_offsets,
                          int num_groups, int rows, int width, int dtype, cudaStream_t stream);

/*
 * The gradient of the expert weights, C = A . B[g]^T for the rows of group g:
 *     d_b[g, n, k] (+)= sum over r in [a_offsets[g], a_offsets[g+1]) of d_c[r, n] * a[r, k]
 * on operands that gmm_quantize_fp8_cols wrote, the scales applied in the tensor core, sums in fp32,
 * one rounding.  Each group has a gradient of its own; a group without rows gets zeros.
 *   d_b: [num_groups, N, K] of `dtype` (GMM_DTYPE_FP32 or GMM_DTYPE_BF16), 16-byte aligned;
 *   accumulate: 1 adds to what d_b holds (GMM_DTYPE_FP32 only), groups without rows untouched;
 *   d_t, d_t_scales: the gradient of C, e4m3 [N, pitch] and uint8 [pitch / 128, N];
 *   a_t, a_t_scales: A, e4m3 [K, pitch] and uint8 [pitch / 128, K], both of
 *   pitch = GMM_FP8_COLS_PITCH(rows, num_groups) and 16-byte aligned (the scales of any);
 *   a_offsets: as gmm_quantize_fp8_cols took them, with the same meaning of bad ones.
 * Requirements: N and K multiples of 16, up to 2^24; num_groups up to 4096; rows below 2^30 + 128
 * (a pitch holds up to 127 rows more than the last whole block).
 * Without rows (rows == 0) the operands and a_offsets may be NULL and are not read.
 * num_groups == 0 launches nothing.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED (a size above its limit,
 * GMM_DTYPE_FP16, 2^31 tiles of 256 x 240, or a device that cannot run CTA pairs), GMM_ERR_CUDA.
 */
int gmm_weight_grad_fp8(gmm_handle_t h, void *d_b, const void *d_t, const void *d_t_scales, const void *a_t,
                        const void *a_t_scales, const uint32_t *a_offsets, int num_groups, int rows, int N, int K,
                        int dtype, int accumulate, cudaStream_t stream);

/*
 * Microscaled 4-bit floating point.  A value is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives) times its block's scale; blocks run along K.
 *   GMM_FP4_NV (nvfp4): blocks of 16, e4m3 scales (sign bit clear), and an optional fp32
 *                       scale of the whole tensor (of each expert's weights).
 *   GMM_FP4_MX (mxfp4): blocks of 32, e8m0 scales (powers of two: 2^(code - 127)).
 * packed: uint8 [rows, K / 2], element k in nibble k % 2 of byte k / 2, low nibble first.
 * scales: uint8 [rows, GMM_FP4_SCALE_PITCH(K, block)]: one byte per block, each row padded to
 * a multiple of 16 bytes.
 */
#define GMM_FP4_NV 0
#define GMM_FP4_MX 1
#define GMM_FP4_SCALE_PITCH(K, block) ((((K) / (block)) + 15) / 16 * 16)

/*
 * Quantise rows of x, optionally gathered:
 *     source row of r: row_slots ? row_slots[r] / top_k : r
 *   nvfp4: s = e4m3(amax / (6 g)), q = e2m1(x / (s g)), g = *global_scale (1 when NULL; it
 *          must be finite and above zero);
 *   mxfp4: s = 2^(floor(log2 amax) - 2), q = e2m1(x / s); global_scale must be NULL;
 * with amax the block's largest magnitude, every step rounded to nearest even in fp32, and
 * saturation at 448 and 6.  s = 0 gives q = 0.  A block that holds an infinity or a NaN gets
 * a NaN scale and zero codes.
 *   packed, scales: as above, 16-byte aligned; padding bytes of a scale row are zeroed;
 *   x: [src_rows, K] of `dtype`, rows x_stride elements apart (0: one row for all);
 *   row_slots: int32 [rows] (gmm_dispatch's row_slots) or NULL; a row with a negative entry
 *   stays untouched, one whose source row is past src_rows too and is reported as
 *   GMM_ERR_BAD_INPUT.
 * Requirements: K a multiple of 32.  rows == 0 launches nothing.
 * Errors (nothing is launched): GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED (K > 2^24),
 * GMM_ERR_CUDA.
 */
int gmm_quantize_fp4(gmm_handle_t h, void *packed, void *scales, const void *x, long long x_stride, int src_rows,
                     const int32_t *row_slots, int top_k, const float *global_scale, int rows, int K, int dtype,
                     int format, cudaStream_t stream);

/*
 * The values that packed and scales stand for: y[r, k] = q * (s * g), of `dtype`, rows
 * y_stride (>= K) elements apart.  The other arguments and the errors are those of
 * gmm_quantize_fp4.
 */
int gmm_dequantize_fp4(gmm_handle_t h, void *y, long long y_stride, const void *packed, const void *scales,
                       const float *global_scale, int rows, int K, int dtype, int format, cudaStream_t stream);

/*
 * The grouped GEMM on microscaled 4-bit operands:
 *     C[r, n] = bf16( ga * gb[e] * sum_k sa[r, k / block] * qa[r, k] * sb[e, n, k / block] * qb[e, n, k] )
 * for the rows and groups of gmm_run, then the optional epilogue; the sums are fp32 on the
 * tensor cores.
 *   a: packed [rows, K / 2]; a_scales [rows, pitch]; b: packed [num_experts, N, K / 2];
 *   b_scales [num_experts, N, pitch] with pitch = GMM_FP4_SCALE_PITCH(K, block), all 16-byte
 *   aligned, both operands of `format`; a_global: fp32, one value, b_global: fp32
 *   [num_experts], each NULL for ones; c and the rest as gmm_run.
 * Requirements: those of gmm_run with K a multiple of 32.  Padding bytes of the scales are
 * not used.  With num_groups == 0 or without rows, c, a and a_scales may be NULL.
 * Errors: as gmm_run_ex, plus GMM_ERR_INVALID_ARG for an unknown format and NULL or
 * misaligned scales, GMM_ERR_UNSUPPORTED where the device cannot run the CTA-pair kernel.
 */
int gmm_run_fp4(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                const void *a_scales, const void *b_scales, int format, const float *a_global, const float *b_global,
                const gmm_epilogue *epilogue, cudaStream_t stream);

/*
 * Allocation-free variant of gmm_run, for callers that cannot call cudaMalloc when
 * they need the GEMM: code running inside an allocator or memory-pool callback, a
 * framework that has reserved all device memory for its own pool, or a runtime that
 * forbids allocations after start-up.  The pages have no counterpart to this call.
 *
 * It computes exactly what gmm_run computes, with the same kernel, on the CALLER'S
 * CURRENT DEVICE (all pointers must live there), and needs no handle: num_experts is
 * passed directly.  The caller still provides every input and output buffer.  The
 * kernel's scratch (a status word and one 2 KB slot of tensor maps per CTA) comes from
 * a fixed array compiled into the library, 524,544 bytes on every GPU that loads it,
 * held until the process exits.  That array has slots for at most 256 CTAs; the grid
 * is one CTA per SM, so a device with more than 256 SMs gets GMM_ERR_UNSUPPORTED.
 *
 * The first call on a device does a one-time set-up (looks up the array's device
 * address, the tensor-map encoder, and the kernel's shared-memory setting); make that
 * first call before any stream capture.  A set-up that fails is not remembered: the
 * next call tries it again.  No call allocates or frees device memory itself, but
 * note that CUDA loads a library's device code lazily by default: the array is
 * reserved on a device when the library's module is first loaded there, which is
 * the first call into this library on that device (this one or any other).  A
 * caller that later hands all free device memory to its own pool should make one
 * call at start-up, before it does so.
 *
 * Every call shares the one array and finds the previous call's contents in it; the
 * call clears the status word itself (stream-ordered on `stream`), rewrites the
 * tensor-map slots, and its kernel returns the array's tile-claim word and
 * finished-CTA counter to zero when it finishes (they are zero when the library is loaded).  Calls whose kernels overlap on the GPU (different streams, or
 * concurrent threads) race on the array: order them on one stream.  The device
 * status (bad offsets / ids) is not reported by this call; the device still applies
 * the same rules (see the header comment).
 * Errors (nothing is launched): those of gmm_run, plus GMM_ERR_INVALID_ARG
 * (num_experts < 1), GMM_ERR_NO_DEVICE (current device is not sm_103),
 * GMM_ERR_UNSUPPORTED (more than 256 SMs, or a device index >= 64).
 */
int gmm_run_noalloc(void *c, const void *a, const uint32_t *a_offsets, const void *b,
                    const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_experts,
                    int num_groups, int N, int K, cudaStream_t stream);

/*
 * The error report of the quantised GEMM page (Modular "multistage_gemm_q", section
 * "Raises": the function raises an error on invalid input) for the conditions that
 * only the device sees: decreasing offsets and out-of-range expert ids, and a
 * kernel that gave up on a pipeline wait.
 * Synchronise `stream`, then read and clear the device status that the kernels of
 * this handle accumulated since the last query.  It speaks for the work that is ordered
 * before it on `stream`: where calls of one handle overlap on several streams, join them
 * first.  What a call on another stream reports meanwhile is in this answer or stays for
 * the next query.  Returns GMM_OK,
 * GMM_ERR_BAD_INPUT or GMM_ERR_DEVICE_TIMEOUT (timeout wins when both are set),
 * or GMM_ERR_CUDA when the synchronisation or the copy fails (for instance after
 * an earlier asynchronous fault).
 */
int gmm_query_status(gmm_handle_t h, cudaStream_t stream);

/* Static, NUL-terminated description of a return code. */
const char *gmm_error_string(int code);

/*
 * Release the handle and its workspace.  The caller must make sure no launch made
 * through the handle is still running (synchronise first).  NULL is accepted.
 */
int gmm_destroy(gmm_handle_t h);

#ifdef __cplusplus
}
#endif

#endif /* GMM_H_ */
