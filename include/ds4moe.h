/*
 * ds4moe -- forward pass of a DeepSeek-V4-style quantized Mixture-of-Experts layer on one
 * NVIDIA GB300 (sm_103a). C ABI: plain pointers and sizes, no C++ or framework types.
 *
 * What one forward computes, for each token x (a row of d bf16 values):
 *
 *   learned routing   z = W_r x + b (fp32), s = sigmoid(z); the top_k experts by
 *                     (s descending, expert index ascending); w_j = s_j / sum of the
 *                     selected s. The bias b (optional) is added before the sigmoid.
 *   table routing     for the first n_hash tokens of a call: experts = table[token id],
 *                     w_j = 1 / top_k (arc PR #89 "expert parallelism stage 0 + stage 1
 *                     (EP=2) for V4's MoE", section "Stage 0": early layers route by a
 *                     fixed token-id table).
 *   routed experts    E_e(x) = W_d (silu(W_g x) * (W_u x)), weights dequantized from
 *                     Q2_K or Q8_0 blocks inside the kernels.
 *   combine           out = sum_j w_j E_{e_j}(x) + S(x): routed terms in ascending expert
 *                     id, then the shared expert S (same SwiGLU form, unscaled), all fp32,
 *                     fixed order, no floating-point atomics, so repeated calls are
 *                     bitwise identical. The plain-sum combine is the one the expert
 *                     parallel page describes (arc PR #89, section "Stage 1 -- EP=2"); its
 *                     bitwise repeatability answers the scheduling-dependent float
 *                     atomicAdd down projection recorded in TrevorS/ds4 PR #13 ("Tested").
 *
 * Tensor mix (ds4 PR #754 "CUDA: add DGX Spark network expert/tensor parallelism", section
 * "Supported paths and safety"): 2-bit Q2_K routed experts, Q8_0 shared expert. Each of
 * routed gate/up, routed down and shared may be either format.
 *
 * Canonical weight bytes accepted by ds4moe_create (little endian). A quantized [R x K]
 * matrix is R rows, each row its K/block blocks back to back; a routed stack is n_experts
 * such matrices back to back.
 *   DS4MOE_FMT_Q8_0: block of 32 weights, 34 bytes = fp16 scale, 32 x int8 q; w = scale*q.
 *   DS4MOE_FMT_Q2_K: super-block of 256 weights, 84 bytes = 16 scale bytes (byte j: low
 *     nibble s_j, high nibble m_j, sub-block j = weights 16j..16j+15), 64 quant bytes
 *     (weight i at byte i>>2, bits 2*(i&3)), fp16 d, fp16 dmin; w_i = d*s_j*q_i - dmin*m_j.
 *
 * Shapes: routed gate/up are [f_routed x d], routed down [d x f_routed], shared gate/up
 * [f_shared x d], shared down [d x f_shared]. Every K dimension must be a multiple of 256
 * for Q2_K and of 128 for Q8_0; d, f_routed and f_shared must be multiples of 128, with
 * d <= 12288 and f_routed, f_shared <= 16384.
 *
 * Error convention: every int-returning call returns DS4MOE_OK (0) or a negative code and
 * records a message readable with ds4moe_last_error() on the calling thread. Device-side
 * faults (none are expected) surface at the caller's next synchronisation.
 */
#ifndef DS4MOE_H
#define DS4MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DS4MOE_OK 0
#define DS4MOE_ERR_INVALID_ARG -1        /* null pointer, bad size or shape */
#define DS4MOE_ERR_UNSUPPORTED_FORMAT -2 /* format enum not Q8_0 / Q2_K, or shape not tileable; also
                                            a Q2_K super-block with |d| >= 0.0666 (more precisely,
                                            15 * 2^16 * |d| >= 65504) on a handle whose max_tokens
                                            needs the batched path (max_tokens > 16 or
                                            max_tokens * top_k > 128): that path dequantizes Q2_K
                                            weights in fp16 as q * 2^-16 times 2^16 * d * s. Handles
                                            with max_tokens <= 16 (and max_tokens * top_k <= 128)
                                            accept any fp16 d: with such scales they serve every
                                            forward on the decode path */
#define DS4MOE_ERR_DEVICE_MISMATCH -3    /* a device pointer lives on another GPU than the handle */
#define DS4MOE_ERR_CAPACITY -4           /* n_tokens > max_tokens given at create */
#define DS4MOE_ERR_OOM -5                /* device allocation failed or exceeded workspace_limit */
#define DS4MOE_ERR_CUDA -6               /* a CUDA runtime call failed */

typedef enum ds4moe_format { DS4MOE_FMT_Q8_0 = 0, DS4MOE_FMT_Q2_K = 1 } ds4moe_format;

typedef struct ds4moe_shapes {
    int32_t d;             /* hidden size */
    int32_t f_routed;      /* routed expert intermediate size */
    int32_t f_shared;      /* shared expert intermediate size (ignored when n_shared == 0) */
    int32_t n_experts;     /* routed experts E, 1..256 */
    int32_t top_k;         /* experts per token, 1..min(E, 16) */
    int32_t n_shared;      /* 0 or 1 always-on shared expert */
    int32_t fmt_gate_up;   /* ds4moe_format of the routed gate and up projections */
    int32_t fmt_down;      /* ds4moe_format of the routed down projection */
    int32_t fmt_shared;    /* ds4moe_format of the shared expert's three projections */
    int32_t has_bias;      /* 1: router_b is read */
    int32_t hash_vocab;    /* rows of the token-id routing table; 0 = no table routing */
    int32_t max_tokens;    /* largest n_tokens of any later forward; sizes the workspace */
    int32_t device;        /* CUDA device ordinal the handle lives on */
    int32_t reserved;
    int64_t workspace_limit; /* bytes; 0 = unlimited. Exceeding it returns DS4MOE_ERR_OOM */
} ds4moe_shapes;

/* Each pointer may be host memory (pageable or pinned) or device memory on shapes.device.
 * ds4moe_create copies and repacks everything; the caller keeps ownership and may free or
 * reuse its buffers as soon as the call returns. */
typedef struct ds4moe_weights {
    const float* router_w;      /* fp32 [E x d] row-major */
    const float* router_b;      /* fp32 [E], read when has_bias, else may be NULL */
    const void* gate;           /* routed gate stack, E x [f_routed x d] canonical blocks */
    const void* up;             /* routed up stack, same shape */
    const void* down;           /* routed down stack, E x [d x f_routed] */
    const void* shared_gate;    /* [f_shared x d], NULL when n_shared == 0 */
    const void* shared_up;      /* [f_shared x d] */
    const void* shared_down;    /* [d x f_shared] */
    const int32_t* hash_table;  /* int32 [hash_vocab x top_k], distinct ids in [0, E) per row (checked
                                   at create: DS4MOE_ERR_INVALID_ARG otherwise); NULL if none */
} ds4moe_weights;

typedef struct ds4moe_stats {
    int32_t n_tokens;          /* tokens of the last forward */
    int32_t distinct_experts;  /* routed experts with at least one token in the last forward */
    int32_t error_flags;       /* device-side conditions of the last forward (0 = none). The
                                  forward itself has already returned DS4MOE_OK when they arise:
                                  read them here after a forward whose result matters.
                                  bit 0: a token id was outside [0, hash_vocab); that token's
                                         routed part was skipped (weights 0), the rest is valid.
                                  bit 2: a pipeline wait of the batched expert GEMM gave up after
                                         its time limit (about one second); the GEMM stopped and
                                         the output rows of that launch are incomplete. One of
                                         bits 17..23 names the wait: 17 weight producer (raw slot
                                         free), 18 activation producer (stage free), 19 dequant
                                         (raw weights landed), 20 dequant (stage free), 21
                                         epilogue (accumulator full), 22 MMA (accumulator free),
                                         23 MMA (stage full).
                                  bit 3: in the batched path, an intermediate |h| = |silu(g) u|
                                         exceeded the fp16 range (65504); it was stored as an
                                         infinity and the affected output rows are not finite.
                                  Other bits are reserved. */
    int32_t reserved;
    int32_t counts[256];       /* tokens per routed expert in the last forward */
} ds4moe_stats;

typedef struct ds4moe_handle ds4moe_handle;

/* Validates shapes, allocates the device weights and a workspace for max_tokens, copies and
 * repacks the weights. Synchronous. On failure *out is set to NULL and nothing leaks.
 * Forwards take one of two paths (same results up to fp32 rounding; both deterministic): the
 * decode path (three kernels, each touched expert read once per token; up to 16 tokens and
 * 128 slots) and the batched path (tensor-core expert GEMMs, each touched expert read once for
 * all its tokens). Forwards of fewer than 8 tokens take the decode path, larger ones the batched
 * path when the handle has it (max_tokens >= 8 and weights within the batched path's Q2_K scale
 * range, see DS4MOE_ERR_UNSUPPORTED_FORMAT). The environment variable DS4MOE_BATCHED_FROM, read
 * here, replaces the 8 (17 keeps every forward the decode kernels can take on the decode path). */
int ds4moe_create(const ds4moe_weights* w, const ds4moe_shapes* s, ds4moe_handle** out);

/* Expert-parallel partial on one GPU (arc PR #89 "expert parallelism stage 0 + stage 1 (EP=2)",
 * section "Stage 1 -- EP=2": a rank holds a subset of the routed experts and computes the sum over
 * its owned slots of w_j E_j(x); the layer output is the plain sum of the ranks' partials).
 * As ds4moe_create, but the handle holds (copies and repacks) only the routed experts
 * owned[0..n_owned): distinct ids in [0, n_experts), in any order, read from host memory during
 * the call; w still describes the full expert stacks. Its forwards route every token over all
 * n_experts exactly as ds4moe_forward does (the router weights and the hash table are whole), and
 * write out = the sum over the token's slots whose expert is held of w_j E_j(x), held terms in
 * ascending expert id, plus S(x) when include_shared is nonzero. With include_shared == 0 the
 * shared expert is neither copied nor run. The partials of handles whose owned sets partition the
 * experts, exactly one of them with include_shared, add up to ds4moe_forward's output up to the
 * fp32 rounding of that sum. ds4moe_get_route returns the whole routing; ds4moe_get_stats counts
 * only the held experts (counts of the others are 0, distinct_experts counts held experts touched).
 * Every block format is sliceable by expert (an expert's matrices are whole), so none is refused
 * here. Errors: DS4MOE_ERR_INVALID_ARG for a NULL owned, n_owned outside 1..n_experts, or an id
 * out of range or named twice; otherwise as ds4moe_create. */
int ds4moe_create_subset(const ds4moe_weights* w, const ds4moe_shapes* s, const int32_t* owned, int32_t n_owned,
                         int32_t include_shared, ds4moe_handle** out);

/* Learned routing for every token. x: device bf16 [n_tokens x d]; out: device fp32
 * [n_tokens x d]; both caller-owned, on the handle's device. stream: a cudaStream_t (NULL =
 * legacy default stream). Asynchronous and stream-ordered: no host synchronisation. A handle
 * serves one stream at a time (its workspace is shared by all calls on it). n_tokens == 0 is
 * a no-op. */
int ds4moe_forward(ds4moe_handle* h, const void* x, int32_t n_tokens, float* out, void* stream);

/* As ds4moe_forward, but tokens 0..n_hash-1 take table routing by token_ids (device int32
 * [n_hash]). n_hash must be 0 when the handle has no table. */
int ds4moe_forward_ex(ds4moe_handle* h, const void* x, int32_t n_tokens, const int32_t* token_ids,
                      int32_t n_hash, float* out, void* stream);

/* As ds4moe_forward_ex with host buffers: copies x (and token_ids) to the device, runs the
 * forward and copies out back, then synchronises the stream before returning. With page-locked
 * host buffers the copies and the kernels replay as one cached CUDA graph (keyed by the token
 * counts and buffer addresses; device forwards cache their kernels' graph the same way), and x and
 * out (when 16-byte aligned) are copied by a kernel that addresses them directly rather than by
 * the copy engines (DS4MOE_SM_COPIES=0 at create turns that off); pageable buffers take separate
 * copies. */
int ds4moe_forward_host(ds4moe_handle* h, const void* x_host, int32_t n_tokens,
                        const int32_t* token_ids_host, int32_t n_hash, float* out_host, void* stream);

/* Copies the last forward's routing to host arrays idx [n_tokens x top_k] and w
 * [n_tokens x top_k] in top-k order (score descending). Synchronises the handle's last
 * stream; meant for tests and measurement, not for a timed path. */
int ds4moe_get_route(ds4moe_handle* h, int32_t* idx_host, float* w_host, int32_t n_tokens);

/* Per-expert token counts, distinct experts touched and error flags of the last forward.
 * Synchronises like ds4moe_get_route. */
int ds4moe_get_stats(ds4moe_handle* h, ds4moe_stats* st);

/* Bytes of device memory the handle holds (weights + workspace). */
int64_t ds4moe_device_bytes(const ds4moe_handle* h);

/* Number of kernel launches one forward of n_tokens learned-routed tokens issues. */
int32_t ds4moe_launches_per_forward(const ds4moe_handle* h, int32_t n_tokens);

/* Per-launch timing for measurement: when enabled, every later forward records a CUDA event
 * after each kernel launch on its stream (this adds event records between launches).
 * ds4moe_get_phase_times waits for the last profiled forward and returns, for each launch in
 * order, its stream time in milliseconds (ms, may be NULL) and a static name (names, may be
 * NULL); *n_phases receives the number of launches (0 when profiling is off). */
int ds4moe_set_profiling(ds4moe_handle* h, int32_t enable);
int ds4moe_get_phase_times(ds4moe_handle* h, float* ms, const char** names, int32_t max_phases,
                           int32_t* n_phases);

/* Routing step alone, allocating nothing (the paper has no counterpart: this is a library
 * convenience). Some callers cannot call cudaMalloc -- an engine that carves its device memory
 * up front and forbids later allocations, a plugin whose host owns the memory budget, a
 * latency-critical path where cudaMalloc may synchronise the device. This call needs no handle:
 * it computes fp32 logits of router_w (device fp32 [n_experts x d]) and router_b (device fp32
 * [n_experts] or NULL) for x (device bf16 [n_tokens x d]), then the sigmoid top-k with ties to
 * the lower index and weights renormalised to sum 1, into idx (device int32
 * [n_tokens x top_k]) and w (device fp32 [n_tokens x top_k]), in top-k order. It computes the
 * same routing as ds4moe_forward with its own kernel (fp32 FMA logits): the fp32 summation order
 * differs from the forward's routers, so logits may differ in the last bits, and the chosen
 * experts agree with the forward's except where the k-th and (k+1)-th scores are within about
 * 1e-6 of each other. Runs on the calling thread's current device, asynchronously on stream.
 * The logits live in a static device array of DS4MOE_NOALLOC_MAX_LOGITS floats that the library
 * image carries (held by every GPU that loads the library until exit): n_tokens * n_experts
 * above that returns DS4MOE_ERR_CAPACITY. The first call on a device looks the array's address
 * up (cudaGetSymbolAddress) and sets the router kernel's attributes in that device's context;
 * make it before any stream capture. All calls on a device share the array, so calls that may
 * overlap on the GPU (unordered streams) race. */
#define DS4MOE_NOALLOC_MAX_LOGITS 262144
int ds4moe_route_noalloc(const float* router_w, const float* router_b, const void* x, int32_t n_tokens,
                         int32_t d, int32_t n_experts, int32_t top_k, int32_t* idx, float* w, void* stream);

/* Test hook of the failure path (no counterpart in the paper: it exists so that the bounded waits
 * of the batched expert GEMM can be shown to end with an error status instead of a hang). The next
 * batched forward of h (more than 16 tokens, or more than 128 routed slots) runs its routed
 * gate/up GEMM with every pipeline wait limited to about 1 ms instead of about 1 s, and the first
 * CTA of that launch withholds one dequant arrival of its K stage `stage` (counted over the CTA's
 * work items). That stage never becomes full, so the MMA's wait for it runs out: the CTA stops,
 * lets its issued copies and MMAs finish, frees its tensor memory and records error bit 2 plus a
 * bit naming the wait (see ds4moe_stats.error_flags); that forward's output is incomplete. The
 * hook applies to one forward and then clears itself. stage >= 0; DS4MOE_ERR_INVALID_ARG
 * otherwise. */
int ds4moe_set_test_stall(ds4moe_handle* h, int32_t stage);

/* Frees everything the handle owns. NULL is allowed. Synchronises the device first. */
void ds4moe_destroy(ds4moe_handle* h);

/* ---------------------------------------------------------------------------------------------
 * Operators on 16-bit matrices: what stands next to the quantized layer in a model whose other
 * weights are kept in bf16 or fp16, and in its training. They need no handle: every operand,
 * result and scratch buffer is the caller's device memory on the calling thread's current device
 * (DS4MOE_ERR_INVALID_ARG for host memory, DS4MOE_ERR_DEVICE_MISMATCH for another GPU's), they
 * allocate nothing, launch asynchronously on `stream`, can be captured in a CUDA graph (the first
 * call of any of them on a device sets its kernels up: make it before a capture), and may run on
 * several streams at once as long as these do not share a workspace. Repeated calls are bitwise
 * identical (fixed summation order, no float atomics).
 *
 * Matrices are row-major; `ld...` is the distance in elements from one row to the next (at least
 * the row's width; 0 means the width itself). Rows need only their element's alignment; operands
 * whose addresses and row distances are multiples of 16 bytes are read by the TMA unit, others by
 * ordinary loads (slower). dtype (DS4MOE_BF16 or DS4MOE_FP16) is the type of all 16-bit operands
 * and results of a call. Products accumulate in fp32 and round once. Results must not overlap
 * inputs except where said. Widths n, k, d and vocab are 1..2^24, rows 0..2^24. */
typedef enum ds4moe_dtype { DS4MOE_BF16 = 0, DS4MOE_FP16 = 1, DS4MOE_FP32 = 2 } ds4moe_dtype;
typedef enum ds4moe_act { DS4MOE_ACT_NONE = 0, DS4MOE_ACT_RELU = 1, DS4MOE_ACT_SILU = 2, DS4MOE_ACT_GELU = 3 } ds4moe_act;

/* Products grouped by expert with ragged sizes. The rows are ordered by group: group g owns rows
 * offsets[g] .. offsets[g+1]-1 (offsets: device int32 [n_groups + 1], non-decreasing, starting at
 * 0 and at most `rows`; n_groups 1..1024; a group may be empty). Group g's weights are
 * W_g = w + g * w_stride, [n x k] with row distance ldw (w_stride 0 means n * ldw).
 *   ds4moe_grouped_mm      y[t]  = W_g x[t]            x [rows x k], y [rows x n]
 *   ds4moe_grouped_mm_dx   dx[t] = W_g^T dy[t]         dy [rows x n], dx [rows x k]
 *   ds4moe_grouped_mm_dw   dW_g  = sum_t dy[t] x[t]^T  dW_g = dw + g * dw_stride, [n x k]; zero for
 *                          an empty group. dw_dtype is dtype or DS4MOE_FP32; accumulate != 0 adds to
 *                          what dw holds.
 * The offsets are read on the device: nothing is synchronised. Offsets out of range are clamped to
 * [0, rows] and a group whose end lies before its start is empty, so that no offsets reach outside the
 * matrices; which rows are computed for decreasing offsets is otherwise unspecified. Rows that belong to no group
 * (from offsets[n_groups] on) are neither read nor written. */
int ds4moe_grouped_mm(const void* x, const void* w, const int32_t* offsets, void* y, int32_t rows, int32_t n,
                      int32_t k, int32_t n_groups, int32_t dtype, int64_t ldx, int64_t ldw, int64_t w_stride,
                      int64_t ldy, void* stream);
int ds4moe_grouped_mm_dx(const void* dy, const void* w, const int32_t* offsets, void* dx, int32_t rows, int32_t n,
                         int32_t k, int32_t n_groups, int32_t dtype, int64_t lddy, int64_t ldw, int64_t w_stride,
                         int64_t lddx, void* stream);
int ds4moe_grouped_mm_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int32_t rows, int32_t n,
                         int32_t k, int32_t n_groups, int32_t dtype, int32_t dw_dtype, int32_t accumulate,
                         int64_t lddy, int64_t ldx, int64_t lddw, int64_t dw_stride, void* stream);

/* Dense product with bias, activation and residual: z = W x + bias, y = act(z) + residual, in fp32,
 * rounded once. x [rows x k], w [n x k], bias [n] or NULL, residual [rows x n] or NULL (it may be y
 * itself), y [rows x n]; zout [rows x n] or NULL receives z rounded to dtype, which the gradient of
 * an activation needs. silu(z) = z / (1 + exp(-z)); gelu is the exact form with erf. */
int ds4moe_linear(const void* x, const void* w, const void* bias, const void* residual, void* y, void* zout,
                  int32_t rows, int32_t n, int32_t k, int32_t act, int32_t dtype, int64_t ldx, int64_t ldw,
                  int64_t ldr, int64_t ldy, int64_t ldz, void* stream);

/* Its gradients, for dy [rows x n]: dz = dy * act'(z), dx = W^T dz [rows x k], dw = sum_t dz[t] x[t]^T
 * [n x k], db = sum_t dz[t] [n] (the residual's gradient is dy itself). z is what zout received (not
 * read, may be NULL, for DS4MOE_ACT_NONE). Each of dx, dw, db may be NULL: it is then not computed (w is
 * read only for dx, x only for dw). Where z is infinite act' is its limit (0 or 1), where it is NaN dz is NaN;
 * where relu is 0 (z <= 0) dz is 0 whatever dy holds. rows == 0 writes zeros into dw and db. dz is rounded to dtype
 * between its computation and the products; db sums the unrounded dz in fp32. workspace: 16-byte
 * aligned device memory of ds4moe_linear_grad_workspace bytes (DS4MOE_ERR_CAPACITY if less). */
int64_t ds4moe_linear_grad_workspace(int32_t rows, int32_t n, int32_t act);
int ds4moe_linear_grad(const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw, void* db,
                       int32_t rows, int32_t n, int32_t k, int32_t act, int32_t dtype, int64_t lddy, int64_t ldx,
                       int64_t ldw, int64_t ldz, int64_t lddx, int64_t lddw, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* Softmax cross entropy of the logits z[t] = W x[t], without storing them: lse[t] = log sum_v exp z[t][v],
 * loss[t] = lse[t] - z[t][labels[t]] (fp32 [rows] each). x [rows x d], w [vocab x d], labels device int32
 * [rows]. A row whose label is ignore_index has loss 0 and no gradient; so has one whose label lies outside
 * [0, vocab), which also sets bit 0 of ds4moe_ops_status. lse is written for every row; it
 * is -inf for a row whose every logit is -inf.
 *   ds4moe_cross_entropy_grad: for dloss (fp32 [rows]) and the lse of the forward,
 *     dz[t][v] = (exp(z[t][v] - lse[t]) - [v == labels[t]]) * dloss[t],
 *     dx[t] = sum_v dz[t][v] W[v], dw[v] = sum_t dz[t][v] x[t], rounded to dtype. Either may be NULL.
 *     The logits are computed again one piece of the vocabulary at a time and dz is rounded to dtype
 *     (relative to the largest finite |dloss|, so that fp16 does not underflow) in the workspace. A dloss
 *     that is not finite makes its own row's dx not finite, and every dw. Rows without a gradient enter dw as zeros
 *     times x: their x has to be finite (padding cleared, not left as it was allocated).
 * workspace: 16-byte aligned device memory. The gradient takes pieces that fit it, of up to 16384
 * words; ds4moe_cross_entropy_workspace returns the bytes that let either call run at full speed. The
 * forward needs 8 bytes per row and 256 words (and 4 per row), the gradient 16 + 4 rows d (rounded up to
 * 16) + 512 (rows rounded up to 8); less returns DS4MOE_ERR_CAPACITY. */
int64_t ds4moe_cross_entropy_workspace(int32_t rows, int32_t vocab, int32_t d);
int ds4moe_cross_entropy(const void* x, const void* w, const int32_t* labels, float* loss, float* lse, int32_t rows,
                         int32_t vocab, int32_t d, int32_t dtype, int32_t ignore_index, int64_t ldx, int64_t ldw,
                         void* workspace, int64_t workspace_bytes, void* stream);
int ds4moe_cross_entropy_grad(const void* x, const void* w, const int32_t* labels, const float* lse,
                              const float* dloss, void* dx, void* dw, int32_t rows, int32_t vocab, int32_t d,
                              int32_t dtype, int32_t ignore_index, int64_t ldx, int64_t ldw, int64_t lddx,
                              int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream);

/* A gated feed-forward block's first half in one kernel, grouped by expert as above: group g's weights W_g are
 * [2n x k], n rows of the gate G_g and then n rows of U_g (w_stride 0 means 2 n ldw), and
 *   h[t] = act(G_g x[t]) * (U_g x[t])        x [rows x k], h [rows x n]; products and act in fp32, rounded once.
 * offsets NULL (n_groups 1): one dense block of all rows. zout [rows x 2n] or NULL receives G_g x[t] and then U_g x[t],
 * rounded to dtype, which the gradient needs. n is 1..2^23. The second half is ds4moe_grouped_mm (ds4moe_linear).
 *   ds4moe_grouped_glu_grad: for dh [rows x n] and z what zout received, a = z's first n columns and b its others,
 *     dz = [dh * b * act'(a), dh * act(a)]  [rows x 2n], required: rounded to dtype, what the products read
 *     dx[t] = W_g^T dz[t]                   [rows x k]
 *     dW_g  = sum_t dz[t] x[t]^T            [2n x k] at dw + g * dw_stride; zero for an empty group
 *   dx and dw may each be NULL (w is read only for dx, x only for dw): ds4moe_grouped_mm_dw takes dz where a gradient in
 *   fp32, or added to an older one, is wanted. dz may be z itself, rows as far apart (else the call is refused). Where act'(a) is 0 the first part of dz is 0 whatever dh and b hold;
 *   act(a) is taken at its limit where a is infinite. rows == 0 writes zeros into dw. */
int ds4moe_grouped_glu(const void* x, const void* w, const int32_t* offsets, void* h, void* zout, int32_t rows, int32_t n,
                       int32_t k, int32_t n_groups, int32_t act, int32_t dtype, int64_t ldx, int64_t ldw,
                       int64_t w_stride, int64_t ldh, int64_t ldz, void* stream);
int ds4moe_grouped_glu_grad(const void* dh, const void* x, const void* w, const int32_t* offsets, const void* z, void* dz,
                            void* dx, void* dw, int32_t rows, int32_t n, int32_t k, int32_t n_groups, int32_t act,
                            int32_t dtype, int64_t lddh, int64_t ldx, int64_t ldw, int64_t w_stride, int64_t ldz,
                            int64_t lddz, int64_t lddx, int64_t lddw, int64_t dw_stride, void* stream);

/* Scores of the logits z[t] = W x[t] at a temperature T (0.001..1000), x [rows x d], w [vocab x d]:
 *   lse[t]        = log sum_v exp(z[t][v] / T)
 *   logprob[t][j] = z[t][tokens[t][j]] / T - lse[t]          tokens device int32 [rows x n_tokens], n_tokens 0..256
 *   entropy[t]    = -sum_v p log p, p = exp(z[t][v] / T - lse[t])
 *   top_index[t], top_logprob[t]: the top_k words with the largest logits, in order, ties to the lower index
 *                                  (int32 and fp32 [rows x top_k], top_k 0..64 and at most vocab)
 * all fp32 but the indices, lists without gaps between rows. The entropy of exact logits is off by about 1e-6 (1 + entropy); the
 * logits' own errors (sums of d products in fp32) count 1 / T times in lse and logprob, up to 2 entropy / T times in it. A place without a token holds -1 and has logprob 0; so has one
 * that lies outside the vocabulary otherwise, which also sets bit 0 of ds4moe_ops_status. lse and entropy may be NULL, the
 * lists where they have no places. A logit of -inf has probability 0; a row with no other has lse -inf, its entropy and
 * log probabilities are NaN. A logit that is NaN makes lse, entropy and the log probabilities of its row NaN and is listed
 * nowhere; places of top_index that this leaves hold -1 and NaN. One of +inf does the same to its row, but is listed.
 * workspace: 16-byte aligned device memory. ds4moe_logprobs_workspace returns the bytes for all rows at once (with top_k the
 * logits in fp32 are in it), and for any smaller number of rows; a call takes the rows in blocks of a multiple of 128 that its workspace holds, each of
 * which reads W (sums may then be joined in another order), and less than a block of 128 (or all) rows needs returns
 * DS4MOE_ERR_CAPACITY. */
int64_t ds4moe_logprobs_workspace(int32_t rows, int32_t vocab, int32_t n_tokens, int32_t top_k);
int ds4moe_logprobs(const void* x, const void* w, const int32_t* tokens, float* logprob, float* lse, float* entropy,
                    int32_t* top_index, float* top_logprob, int32_t rows, int32_t vocab, int32_t d, int32_t n_tokens,
                    int32_t top_k, int32_t dtype, float temperature, int64_t ldx, int64_t ldw, void* workspace,
                    int64_t workspace_bytes, void* stream);

/* Distillation from a teacher's top logits, the student's logits z[t] = W x[t] not stored. Row t has top_k entries (1..256):
 * words ids[t][j] (device int32 [rows x top_k]; -1: no entry) with the teacher's logits teacher[t][j] (fp32, before the
 * temperature; log probabilities do as well). With p = softmax over the row's entries of teacher / T and
 * q = softmax over the vocabulary of z / T:
 *   loss[t] = sum_j p_j (log p_j - logq[t][j]), logq[t][j] = z[t][ids[t][j]] / T - lse[t], lse as above (fp32, all written;
 *   logq is 0 without an entry). A word named twice counts with both its entries. A row without entries, or with none above
 *   -inf, has loss 0 and no gradient; an id other than -1 outside the vocabulary is no entry and sets bit 0 of
 *   ds4moe_ops_status. A teacher logit of +inf or NaN makes its row's loss NaN.
 *   ds4moe_distill_grad: for dloss (fp32 [rows]) and the lse and logq of the forward,
 *     dz[t][v] = (q_v - sum over the entries that name v of p_j) * dloss[t] / T, dx[t] = sum_v dz[t][v] W[v],
 *     dw[v] = sum_t dz[t][v] x[t], rounded to dtype. Either may be NULL. dz, the pieces of the vocabulary and what is not
 *     finite are as for ds4moe_cross_entropy_grad.
 * T is not applied to the loss once more (a caller who wants T^2 has it in dloss). workspace: as for the cross entropy;
 * ds4moe_distill_workspace returns the bytes that let either call of so many rows, or of fewer, run at full speed (pieces of
 * 16384 words, and for up to 512 rows of as many as take 64 MB, or the vocabulary). The forward takes the rows in blocks as
 * ds4moe_logprobs does; the gradient needs 16 + 4 rows (d + 1 + top_k) + 512 (rows rounded up to 8) and 48 for rounding. */
int64_t ds4moe_distill_workspace(int32_t rows, int32_t vocab, int32_t d, int32_t top_k);
int ds4moe_distill(const void* x, const void* w, const int32_t* ids, const float* teacher, float* loss, float* lse,
                   float* logq, int32_t rows, int32_t vocab, int32_t d, int32_t top_k, int32_t dtype, float temperature,
                   int64_t ldx, int64_t ldw, void* workspace, int64_t workspace_bytes, void* stream);
int ds4moe_distill_grad(const void* x, const void* w, const int32_t* ids, const float* teacher, const float* lse,
                        const float* logq, const float* dloss, void* dx, void* dw, int32_t rows, int32_t vocab, int32_t d,
                        int32_t top_k, int32_t dtype, float temperature, int64_t ldx, int64_t ldw, int64_t lddx,
                        int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream);

/* Device-side conditions of the 16-bit operators on the current device since the last call of this
 * function: synchronises the device, copies the flags to the host word and clears them. bit 0: a label, token or id
 * outside the vocabulary; bit 2: a pipeline wait gave up after its time limit (about one second) and the
 * results of that call are incomplete. One of bits 17..23 names the wait: 17 loads (stage free), 18 the
 * clearing of a ragged end (stage loaded), 21 epilogue (accumulator full), 22 MMA (accumulator free), 23 MMA
 * (stage loaded). */
int ds4moe_ops_status(int32_t* flags);

/* Message of the last failed call on this thread ("" if none). */
const char* ds4moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DS4MOE_H */
