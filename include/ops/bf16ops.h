/*
 * bf16ops.h -- C ABI of libbf16ops: the operators on either side of the weight sync.
 *
 * libbf16delta (bf16delta.h) moves a trainer's new BF16 weights to the rollout workers.  This
 * library holds what makes those weights and what answers with them:
 *
 *   AdamW over many tensors at once (bo_adamw_*): the optimizer step whose result the compress
 *   encodes, with first and second moments in 32 or in 8 bits, an FP32 master copy or BF16
 *   weights alone, the global gradient norm, and clipping by it.
 *
 *   Low-rank adapters of many requests (bo_adapter_*): forward and backward beside a projection
 *   that all requests share.  The factors are read where they lie, so a delta applied to them
 *   (bd_decompress) takes effect with the next call.
 *
 *   Token log probabilities (bo_logprobs_*): what a worker reports beside its answers and a
 *   trainer's loss is made of, with the distribution's entropy and its top alternatives, and the
 *   logits' gradient.
 *
 *   Routing to experts (bo_routing_*): the experts of each token of a mixture and their weights,
 *   per-expert counts and the balance loss, and the gradient of the router's logits.
 *
 * Conventions are those of bf16delta.h: "d_" pointers are device memory and "h_" pointers host
 * memory, all owned by the caller; nothing is allocated; calls are asynchronous on `stream` and
 * never wait for the GPU; the return value (a bd_status) reports argument and launch errors
 * only, and nothing has been enqueued when it is BD_ERR_INVALID_ARG.  Every call may be captured
 * in a CUDA graph.  Handles (bo_adamw, bo_adapter_set, bo_adapter_rows, bo_logprobs, bo_routing) are plain structs in host
 * memory: the caller owns them and may copy or drop them; their fields are the library's.  A handle
 * belongs to the device that was current when it was made; with another one current, calls that
 * take it return BD_ERR_INVALID_ARG.
 */
#ifndef BF16OPS_H
#define BF16OPS_H

#include <stdint.h>

#include "bf16delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status beside those of bd_status: the step was skipped because the gradient norm was
 * not finite; weights, master, moments and the step count are as before the call. */
#define BO_SKIPPED_NONFINITE 16

/* ------------------------------------------------------------------------------- AdamW
 *
 * For every element, with t the number of this step (1 for the first):
 *   c = min(1, max_norm / (norm + 1e-6)) when clipping, else 1;   g' = c g
 *   m = beta1 m + (1 - beta1) g'          v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr wd) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * computed in FP32, where v may underflow to 0 under an m that did not: with eps = 0 the quotient is
 * 0 wherever its denominator is.  norm = sqrt(sum of g^2 over all tensors), summed in a fixed order
 * (in FP32 too: a gradient above 1.8e19 has an infinite square, and the norm is not finite then).
 *
 * State arenas.  The elements of item i take the blocks of 256 from first_block on (the last
 * one padded); m, v and master of all items lie in one arena each, indexed by
 * 256 * block + element.  Padding is never read into a result and stays as it is (8-bit codes
 * of padding are written as 0).
 *
 * 8-bit moments: per block an FP32 scale (sm = max |m|, sv = max v) and codes
 *   m: int8 c, value sign(c) (c/127)^2 sm, c = rint(127 sqrt(|m| / sm)) with m's sign;
 *   v: uint8 c, value (c/255)^4 sv; of the two codes whose values enclose v the upper one with
 *      the probability (v - lower) / (upper - lower), and never 0 for v > 0.
 * The codes are spaced so that small values keep relative precision.  v is rounded
 * stochastically because beta2 moves it by less than half a code step: rounded to nearest it
 * would stay where it is.  A block that holds a value that is not finite gets a NaN scale and
 * reads as NaN throughout (pass max_norm, if only INFINITY, to skip such steps).
 *
 * Random bits: R_j = mix64(mix64(seed ^ t G) + (j + 1) G) with SplitMix64's mix64 and G
 * (bf16delta.h) and j = e >> 1 for arena element e, whose 32 bits are R_j >> 32 * (e & 1); the
 * upper 16 round v's code, the lower 16 a BF16 weight.  A step is a function of its inputs,
 * the seed and t. */

typedef enum bo_weight_kind {
  BO_WEIGHT_MASTER = 0, /* FP32 master in the arena; d_out gets its BF16 rounding */
  BO_WEIGHT_BF16 = 1,   /* BF16 weights alone: d_weight is read, d_out written */
  BO_WEIGHT_FP32 = 2    /* FP32 weights: d_weight is read, d_out written */
} bo_weight_kind;

typedef enum bo_dtype { BO_BF16 = 0, BO_FP32 = 1 } bo_dtype;

#define BO_BLOCK_ELEMS 256u
#define BO_ADAMW_STOCHASTIC 1u /* flag: BF16 weights alone are rounded stochastically */

/* One tensor of a step.  Pointers 16-byte aligned. */
typedef struct bo_adamw_item {
  const void* d_weight;  /* weights before the step (not read, may be NULL, with a master) */
  void* d_out;           /* weights after the step; == d_weight for a step in place */
  const void* d_grad;    /* gradients */
  uint64_t n;            /* elements */
  uint64_t first_block;  /* first block of 256 in the arenas */
  float weight_decay;
  uint32_t reserved;     /* 0 */
} bo_adamw_item;

/* The arenas (256-byte aligned), of `blocks` blocks each. */
typedef struct bo_adamw_state {
  void* d_m;            /* float, or int8 codes */
  void* d_v;            /* float, or uint8 codes */
  float* d_m_scale;     /* 8 bits only: one per block */
  float* d_v_scale;
  float* d_master;      /* BO_WEIGHT_MASTER only */
  uint64_t blocks;
} bo_adamw_state;

/* Results of a step on the device. */
typedef struct bo_adamw_control {
  int64_t step;         /* steps taken */
  float norm;           /* gradient norm of the last step (when max_norm was given) */
  float coef;           /* its clipping factor */
  int32_t status;       /* BD_OK or BO_SKIPPED_NONFINITE */
  uint32_t ticket[3];   /* the library's */
} bo_adamw_control;

typedef struct bo_adamw {
  bo_adamw_state state;
  bo_adamw_control* d_control;
  void* d_chunks;
  double* d_partials;
  uint64_t chunks;
  uint32_t weight_kind, grad_dtype, state_bits, flags;
  int32_t device;
} bo_adamw;

/* Arguments of one step. */
typedef struct bo_adamw_step_args {
  float lr;
  const float* d_lr;    /* when not NULL, the rate is read from here instead */
  double beta1, beta2;
  float eps;
  float max_norm;       /* > 0: clip, and skip a step whose norm is not finite; 0: neither */
  uint64_t seed;
} bo_adamw_step_args;

/* Bytes of device memory (256-byte aligned) that a plan over k tensors takes; 0 on bad
 * arguments. */
BD_API uint64_t bo_adamw_plan_size(const bo_adamw_item* h_items, uint32_t k);

/* Lays the tensor table out in d_plan and fills *h_out.  h_items is read during the call only.
 * step: steps taken so far.  The tensors, the arenas and d_plan must stay where they are while
 * the handle is used.  What a step writes (outputs, arenas, d_plan) may not overlap anything else of
 * the plan, but for an output that is its own item's weights, nor may the items' blocks: a tensor that
 * two items share is refused. */
BD_API int bo_adamw_plan(const bo_adamw_item* h_items, uint32_t k, const bo_adamw_state* state,
                         uint32_t weight_kind, uint32_t grad_dtype, uint32_t state_bits,
                         uint32_t flags, int64_t step, void* d_plan, uint64_t plan_bytes,
                         bo_adamw* h_out, void* stream);

/* One step over all tensors of the plan. */
BD_API int bo_adamw_step(const bo_adamw* h, const bo_adamw_step_args* args, void* stream);

/* The global gradient norm alone: control.norm, and control.coef for max_norm (1 for 0). */
BD_API int bo_adamw_norm(const bo_adamw* h, float max_norm, void* stream);

/* Both moments of an 8-bit state as values of `dtype`, in the arenas' layout (256 * blocks
 * elements each; 16-byte aligned).  Either output may be NULL. */
BD_API int bo_adamw_moments(const bo_adamw* h, uint32_t dtype, void* d_m, void* d_v,
                            void* stream);

/* ------------------------------------------------------------------- low-rank adapters
 *
 * Row t of a batch belongs to adapter a(t), or to none.  With the adapter's factors
 * A (rank x hidden) and B (out x rank) and its scale s:
 *   forward    low[t] = s A x[t]            y[t] += B low[t]
 *   backward   dlow[t] = s B^T dy[t]        dx[t] += A^T dlow[t]
 *              dA = sum over its rows of dlow[t] x[t]^T
 *              dB = sum over its rows of dy[t] low[t]^T
 * y is the output of the projection that all rows share (and dx that projection's part of the
 * gradient): both are updated in place, so adapter rows cost one read and one write of them.
 * Rows without an adapter are neither read nor written.  Sums are held in FP32; low and dlow
 * are rounded to BF16, the type of the tensor cores' operands, once per row and rank (an error
 * of at most 2^-8 of each term, that of a model that stores its low-rank activations); every output is
 * rounded once.  With few rows the product with low takes it as two BF16 numbers, its rounding and
 * what that cut off.  An infinity in x, dy, y or dx gives what the formula gives for its row, and a
 * low beyond BF16's largest number counts as infinity; an infinity in a factor gives infinity or NaN
 * where it enters.
 * A row's result does not depend on which other rows are in the batch, nor on their order.  It may
 * depend on the numbers of rows and adapters, which choose the form (low in one BF16 number or in
 * two) and where its sums are cut: batches of other sizes can differ in the last bits.  Every sum has
 * one order for given numbers of rows of each adapter, so that the same call repeats its results.
 *
 * x, y, dy, dx: rows of BF16 with a row stride in elements; any sizes and strides (16-byte
 * aligned rows, with hidden and out multiples of 8, take wide accesses). */

#define BO_ADAPTER_MAX_RANK 128u
#define BO_ADAPTER_MAX_COUNT 65535u   /* adapters of a set */
#define BO_ADAPTER_MAX_WIDTH (1u << 24)
#define BO_ADAPTER_MAX_ROWS (1u << 30)

/* One adapter.  Row strides in elements: at least hidden for down, at least rank for up.  The
 * gradients are NULL in all adapters of a set (a backward pass then gives dx alone) or in none.  A
 * gradient may not overlap another one or a factor of the set (refused), nor anything else of a
 * backward call.  Adapters may share factors, but not gradients. */
typedef struct bo_adapter {
  const uint16_t* d_down;  /* A: rank x hidden */
  const uint16_t* d_up;    /* B: out x rank */
  uint64_t ld_down, ld_up;
  void* d_grad_down;       /* dA, dB: as A and B, of grad_dtype */
  void* d_grad_up;
  uint64_t ld_grad_down, ld_grad_up;
  uint32_t rank;           /* 1 to BO_ADAPTER_MAX_RANK */
  float scale;
} bo_adapter;

/* A set of adapters of one projection, laid out by bo_adapter_set_init. */
typedef struct bo_adapter_set {
  const void* d_table;
  uint32_t k, hidden, out;
  uint32_t rank;           /* columns of low: the largest rank, as 16, 32, 64 or 128 */
  uint32_t grad_dtype, has_grads, wide;
  int32_t device;
} bo_adapter_set;

/* For tests of the kernels' bounded waits: set in bo_adapter_set.wide, it keeps the first stage of
 * the forms on the tensor cores' own memory from ever being reported, so that their waits run out (two
 * seconds each) and the calls set *d_status. */
#define BO_ADAPTER_DEBUG_STALL 0x80000000u

/* The rows of a batch grouped by adapter, laid out by bo_adapter_rows_init. */
typedef struct bo_adapter_rows {
  const int32_t* d_perm;     /* rows, grouped */
  const int32_t* d_offsets;  /* adapter a has d_perm[d_offsets[a] .. d_offsets[a + 1]) */
  const int32_t* d_blocks;   /* blocks of 64 rows (counted as at least four) of the adapters before */
  const void* d_tiles[3];    /* tiles of at most 16, 64 and 128 rows of one adapter */
  const int32_t* d_ntiles;   /* how many of each */
  int32_t* d_status;         /* as given; BD_ERR_CUDA from a call whose waits ran out (its outputs
                                are not to be used), until the rows are grouped again */
  uint32_t rows, k;
  int32_t device;
} bo_adapter_rows;

/* Bytes of device memory (256-byte aligned) for a set of k adapters. */
BD_API uint64_t bo_adapter_set_size(uint32_t k);

/* Lays out the table of k adapters (read during the call only).  The factors and gradients
 * must stay where they are; their values may change between calls. */
BD_API int bo_adapter_set_init(const bo_adapter* h_items, uint32_t k, uint32_t hidden,
                               uint32_t out, uint32_t grad_dtype, void* d_set,
                               uint64_t set_bytes, bo_adapter_set* h_out, void* stream);

/* Bytes of device memory (256-byte aligned) to group `rows` rows over k adapters. */
BD_API uint64_t bo_adapter_rows_size(uint32_t rows, uint32_t k);

/* Groups rows by adapter on the device: d_index[t] is row t's adapter, -1 for none.  An index
 * outside -1 .. k - 1 sets *d_status (optional) to BD_ERR_INVALID_ARG, else BD_OK, and counts
 * as none.  One grouping serves every projection of a model step.  The call reads d_index in
 * stream order; calling it again on the same memory regroups for new values. */
BD_API int bo_adapter_rows_init(const int32_t* d_index, uint32_t rows, uint32_t k, void* d_rows,
                                uint64_t rows_bytes, bo_adapter_rows* h_out, int32_t* d_status,
                                void* stream);

/* y += the adapters' products, in place.  d_low receives low, which the backward pass takes:
 * `rows` rows of set->rank columns, 16-byte aligned; columns past an adapter's rank are written
 * as 0, rows without an adapter not at all.  It may be NULL below bo_adapter_low_rows(set) rows;
 * from there on the call needs it as its workspace. */
BD_API int bo_adapter_forward(const bo_adapter_set* set, const bo_adapter_rows* rows,
                              const uint16_t* d_x, uint64_t ldx, uint16_t* d_y, uint64_t ldy,
                              uint16_t* d_low, void* stream);

/* The number of rows from which bo_adapter_forward needs d_low (0: not a set). */
BD_API uint32_t bo_adapter_low_rows(const bo_adapter_set* set);

/* Bytes of workspace (256-byte aligned) that bo_adapter_backward takes. */
BD_API uint64_t bo_adapter_backward_workspace_size(const bo_adapter_set* set, uint32_t rows);

/* dx += (in place; d_dx may be NULL) and, when the set has gradients, dA and dB of every
 * adapter (0 for one without rows), written over what is there or, with accumulate, added to
 * it.  d_low is the forward pass's. */
BD_API int bo_adapter_backward(const bo_adapter_set* set, const bo_adapter_rows* rows,
                               const uint16_t* d_x, uint64_t ldx, const uint16_t* d_dy,
                               uint64_t lddy, const uint16_t* d_low, uint16_t* d_dx,
                               uint64_t lddx, int32_t accumulate, void* d_ws, uint64_t ws_bytes,
                               void* stream);

/* --------------------------------------------------------------- token log probabilities
 *
 * Row t holds the logits x_j of `vocab` tokens; v is its given token and T its temperature:
 *   z_j = x_j / T        lp_j = z_j - ln sum_i e^(z_i)        p_j = e^(lp_j)
 *   logprob = lp_v       entropy H = -sum_j p_j lp_j
 *   top: the `top` tokens of greatest x_j in order, of equal ones the lowest first, and their lp_j
 * and, from the gradients g of logprob and h of the entropy,
 *   dx_j = (g ([j = v] - p_j) - h p_j (lp_j + H)) / T
 * computed in FP32 from logits of BF16 or FP32, by differences from the row's greatest logit: lp_j =
 * (x_j - max) / T - ln sum_i e^((x_i - max) / T), whose error does not depend on where the row lies.
 *
 * A row whose token is negative is left out: it is not read, its logprob, entropy and
 * top_logprobs are 0, its top tokens -1 and its gradient 0.  A token of `vocab` or more, and a
 * temperature that is not a positive number, make the row's logprob and gradient NaN.  A logit of
 * -infinity is a token of probability 0, which adds nothing to the entropy.  A row of nothing else
 * has no distribution: logprob and top_logprobs are -infinity, entropy and gradient 0.  A NaN or
 * +infinity in a row makes its logprob, entropy and gradient NaN; NaN counts as the greatest among
 * the top tokens.  Rows whose g and h are both 0 have the gradient 0 and are not read.
 *
 * Sums have one order for given sizes and alignment, so the same call repeats its results. */

#define BO_LOGPROBS_MAX_TOP 32u
#define BO_LOGPROBS_MAX_VOCAB (1u << 24)
#define BO_LOGPROBS_MAX_ROWS (1u << 28)

/* Results of up to `rows` rows, and what the backward pass takes from the forward one.  Rows behind
 * those of a call stay as they were. */
typedef struct bo_logprobs {
  float* d_logprobs;      /* rows */
  float* d_entropy;       /* rows; NULL where it was not asked for */
  float* d_top_logprobs;  /* rows x top */
  int32_t* d_top_tokens;  /* rows x top */
  void* d_saved;          /* the library's */
  uint32_t rows, vocab, top;
  int32_t device;
} bo_logprobs;

/* Bytes of device memory (256-byte aligned) for the results; 0 on bad arguments.  top is at most
 * vocab and BO_LOGPROBS_MAX_TOP; entropy is 0 or 1. */
BD_API uint64_t bo_logprobs_size(uint32_t rows, uint32_t vocab, uint32_t top, uint32_t entropy);

/* Lays the results out in d_mem and zeroes them (in the stream's order). */
BD_API int bo_logprobs_init(uint32_t rows, uint32_t vocab, uint32_t top, uint32_t entropy,
                            void* d_mem, uint64_t mem_bytes, bo_logprobs* h_out, void* stream);

/* Log probabilities of d_tokens (int32 or int64 by token_bytes, 4 or 8) in the first `rows` rows.
 * d_logits: rows of `vocab` values with a row stride of ld elements.  Strides of tokens and
 * temperatures are in elements and may be 0.  d_temperature: one number a row, or NULL for
 * `temperature` throughout (a positive number). */
BD_API int bo_logprobs_forward(const bo_logprobs* h, const void* d_logits, uint32_t dtype,
                               uint64_t ld, uint32_t rows, const void* d_tokens,
                               uint32_t token_bytes, uint64_t token_stride, float temperature,
                               const float* d_temperature, uint64_t temperature_stride,
                               void* stream);

/* The logits' gradient for the forward call before it on this handle, over the same logits and no
 * more rows than it had: written to d_grad_logits, of the logits' type, with a row stride of ld_grad
 * elements.  That may be the logits themselves (with the same stride), which the gradient then takes
 * the place of, but may not overlap anything else of the call.  Of d_grad_logprobs and d_grad_entropy
 * one may be NULL (0 throughout); strides in elements, 0 for one number for all rows.  d_grad_entropy
 * needs a handle with entropy. */
BD_API int bo_logprobs_backward(const bo_logprobs* h, const void* d_logits, uint32_t dtype,
                                uint64_t ld, uint32_t rows, const float* d_grad_logprobs,
                                uint64_t grad_logprobs_stride, const float* d_grad_entropy,
                                uint64_t grad_entropy_stride, void* d_grad_logits,
                                uint64_t ld_grad, void* stream);

/* -------------------------------------------------------------------- routing to experts
 *
 * Token t's router logits x_e over `experts` experts:
 *   p = softmax(x)       the k experts of greatest x_e in order, of equal ones the lowest first
 *   weight of the i-th chosen:  w_i = p_i, or normalized  w_i = p_i / (sum over the chosen)
 *   n_e: tokens that chose e;  N: tokens;  f_e = n_e / (N k);  P_e = (sum over tokens of p_e) / N
 *   balance loss L = experts * sum_e f_e P_e     (1 when all are alike)
 * and, from the gradients of the weights and of L (n_e has none, so dL/dp_te = experts f_e / N),
 * the gradient of x.  Computed in FP32 from logits of BF16 or FP32; each output is rounded once.
 *
 * Tokens that the mask leaves out, and tokens whose logits are all -infinity, are not counted: their
 * experts are -1, their weights and gradients 0.  A single logit of -infinity is an expert of
 * probability 0, chosen only where fewer than k others are left.  A NaN or +infinity makes the
 * token's weights and gradient NaN, and with them P and L; NaN counts as the greatest.
 *
 * Sums have one order for given sizes, so the same call repeats its results.  A token's experts and
 * normalized weights do not depend on the call's other tokens; weights that are not normalized are divided
 * by a sum over all experts, whose order, and so the weights' last bits, may change with the number of
 * tokens. */

#define BO_ROUTING_MAX_EXPERTS 1024u
#define BO_ROUTING_MAX_K 32u
#define BO_ROUTING_MAX_TOKENS (1u << 28)

/* Results of up to `tokens` tokens.  Weights and experts of tokens behind those of a call stay as
 * they were. */
typedef struct bo_routing {
  float* d_weights;       /* tokens x k */
  int32_t* d_experts;     /* tokens x k */
  int32_t* d_counts;      /* n: experts */
  float* d_probs;         /* P: experts */
  float* d_loss;          /* L */
  int32_t* d_real;        /* N */
  void* d_partials;       /* the library's */
  uint32_t tokens, experts, k, normalize;
  int32_t device;
} bo_routing;

/* Bytes of device memory (256-byte aligned) for the results; 0 on bad arguments.  k is at most
 * experts and BO_ROUTING_MAX_K. */
BD_API uint64_t bo_routing_size(uint32_t tokens, uint32_t experts, uint32_t k);

/* Lays the results out in d_mem and zeroes them (in the stream's order).  normalize is 0 or 1. */
BD_API int bo_routing_init(uint32_t tokens, uint32_t experts, uint32_t k, uint32_t normalize,
                           void* d_mem, uint64_t mem_bytes, bo_routing* h_out, void* stream);

/* Routes the first `tokens` tokens.  d_logits: rows of `experts` values with a row stride of ld
 * elements.  d_mask: NULL, or a byte per token, 0 to leave it out, with a stride in bytes. */
BD_API int bo_routing_forward(const bo_routing* h, const void* d_logits, uint32_t dtype,
                              uint64_t ld, uint32_t tokens, const uint8_t* d_mask,
                              uint64_t mask_stride, void* stream);

/* The logits' gradient for the forward call before it on this handle, over the same logits and no
 * more tokens than it had, with the experts and counts as they are in its results (a number there that is
 * no expert's counts as none).  d_grad_weights: the weights' gradients (NULL: 0), with strides in
 * elements of tokens and of choices, which may be 0.  The gradient of L is *d_grad_loss, or
 * grad_loss where that is NULL.  d_counts: n to take in place of the handle's (NULL), as of several
 * batches together; f is n over its sum.  d_grad_logits: as in bo_logprobs_backward. */
BD_API int bo_routing_backward(const bo_routing* h, const void* d_logits, uint32_t dtype,
                               uint64_t ld, uint32_t tokens, const float* d_grad_weights,
                               uint64_t grad_stride, uint64_t grad_choice_stride, float grad_loss,
                               const float* d_grad_loss, const int32_t* d_counts,
                               void* d_grad_logits, uint64_t ld_grad, void* stream);

/* Library utility: static description of a status, bd_status included. */
BD_API const char* bo_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* BF16OPS_H */
