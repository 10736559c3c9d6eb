/*
 * ep_moe.h -- C ABI of libep_amd.so, second part: what stands on both sides
 * of the token shuffle of ep.h on one MI355X (gfx950).
 *
 *   ep_gate             router scores -> topk_idx, topk_weights (what every
 *                       call of ep.h takes), and ep_gate_backward, its
 *                       gradient
 *   ep_matvec           products of a few rows with one weight matrix
 *   ep_expert_matvec    products of the received rows of a dispatch with
 *                       their experts' matrices (between ep_dispatch and
 *                       ep_combine)
 *   ep_matmul,          the same in 8-bit integers on both sides, for any
 *   ep_expert_matmul    number of rows: rows as an int8 dispatch delivers
 *                       them, with a scale for each row and each output;
 *                       ep_matmul_split, with a workspace, is faster for
 *                       few rows of many columns
 *   ep_moe_layer        the whole expert layer for a few tokens, from
 *                       topk_idx to the combined output, without the shuffle
 *   ep_balance_loss     per-expert counts of a routing and the balance loss,
 *                       and ep_balance_loss_backward, its gradient
 *
 * The conventions of ep.h hold for every call: d_* are device pointers of
 * the current HIP device, the caller owns all memory, `stream` is a
 * hipStream_t, calls are stream-ordered and asynchronous and may be captured
 * into a HIP graph, invalid arguments are rejected on the host before any
 * HIP call, and ep_last_error_message() gives the reason.
 */
#ifndef EP_AMD_EP_MOE_H
#define EP_AMD_EP_MOE_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- router ------------------------------------------------------------ */

enum {
    EP_SCORE_SOFTMAX = 0,   /* s = softmax(logits) over all eligible experts   */
    EP_SCORE_SIGMOID = 1    /* s = sigmoid(logits), each expert by itself      */
};

/* Element type of the logits (and of their gradient). */
enum { EP_LOGITS_FP32 = 0, EP_LOGITS_BF16 = 1 };

typedef struct ep_gate_config {
    int32_t num_experts;   /* E: 1..1024                                       */
    int32_t num_topk;      /* K: 1..16, at most E                              */
    int32_t scoring;       /* EP_SCORE_*                                       */
    int32_t renormalize;   /* 1: weights divided by their sum                  */
    int32_t num_groups;    /* 0 or 1: none.  G > 1: group-limited gating, the
                              experts in G equal contiguous groups, G <= 64    */
    int32_t topk_groups;   /* groups a token may use, 1..G                     */
    int32_t group_top;     /* a group's score is the sum of its best this many
                              choice values, 1..E/G                            */
    int32_t group_limit;   /* 1: a token takes only those group_top experts of
                              a group it uses; 0: any expert of it             */
    int32_t logits_type;   /* EP_LOGITS_*                                      */
    float scale;           /* the weights' factor, finite                      */
} ep_gate_config;

/* Chooses K experts for each of num_tokens tokens.
 *   d_logits [num_tokens, E]; d_bias fp32 [E] or NULL: added to the scores for
 *   the choice only (a balancing bias), never to the weights; d_token_mask
 *   uint8 [num_tokens] or NULL: tokens with 0 (padding) get no expert.
 *   choice[e] = s[e] + bias[e].  With groups only the topk_groups groups of the
 *   highest score keep their experts.  The K experts of the highest choice are
 *   listed highest first; ties, of groups too, go to the lower id.
 *   d_topk_idx int32 [num_tokens, K]; d_topk_weights fp32 [num_tokens, K]:
 *   w = scale * s[idx], divided by the chosen s' sum with renormalize.
 *   Choices are exact: scores that two experts' order could hang on are
 *   compared in 64 bits (without a bias, by their logits).
 *   An expert whose logit is NaN or -infinity, or whose choice is, is not
 *   eligible; a logit of +infinity counts as the largest finite fp32.  Entries
 *   for which no eligible expert is left are -1 with weight 0.
 *   EP_ERR_INVALID_ARG if the groups cannot hold K experts. */
ep_status ep_gate(const ep_gate_config* cfg, const void* d_logits, const float* d_bias,
                  const uint8_t* d_token_mask, int64_t num_tokens, int32_t* d_topk_idx,
                  float* d_topk_weights, void* stream);

/* Gradient of ep_gate's weights with respect to the logits, the choice held
 * fixed (the bias and the mask only act on the choice and have none):
 *   d_grad_logits [num_tokens, E], of the logits' type, written whole.
 *   d_topk_idx: ep_gate's, or any; ids outside [0, E) are masked entries: their
 *   gradient is not read and they take no share of the normalisation.  An id
 *   listed twice counts twice.  Sums are in fp32. */
ep_status ep_gate_backward(const ep_gate_config* cfg, const void* d_logits,
                           const int32_t* d_topk_idx, const float* d_grad_weights,
                           int64_t num_tokens, void* d_grad_logits, void* stream);

/* ---- balance loss --------------------------------------------------------- */

typedef struct ep_balance_config {
    int32_t num_experts;   /* E: 1..1024                                       */
    int32_t num_topk;      /* K: 1..16, at most E                              */
    int32_t scoring;       /* EP_SCORE_*                                       */
    int32_t normalize;     /* sigmoid: 1 = divided by their sum over all experts;
                              a softmax is so in any case                      */
    int32_t logits_type;   /* EP_LOGITS_*                                      */
    float coefficient;     /* of the loss, finite                              */
} ep_balance_config;

/* Sequences of one call, at most. */
#define EP_BALANCE_MAX_SEQUENCES (1 << 18)

/* Bytes of device workspace that ep_balance_loss needs. */
ep_status ep_balance_workspace_size(const ep_balance_config* cfg, int64_t num_tokens,
                                    int64_t num_sequences, int64_t* bytes);

/* Counts of a routing and the loss that keeps experts evenly used.  With V_q the
 * unmasked tokens of sequence q, T_q their number and p their scores:
 *   d_counts int32 [Q, E]: entries of V_q's topk_idx rows that name the expert;
 *   d_seq_tokens int32 [Q]: T_q;
 *   d_score_sums fp32 [Q, E]: sum over V_q of p[t, e];
 *   d_loss fp32 [1]: coefficient / Q * sum over q with T_q > 0 of
 *     E / (K * T_q^2) * sum over e of counts[q, e] * score_sums[q, e],
 *   coefficient for a sequence that uses its experts evenly.
 *   d_logits [num_tokens, E]; d_topk_idx int32 [num_tokens, K], ep_gate's or any:
 *   ids outside [0, E) are not counted, an id listed twice counts twice;
 *   d_token_mask uint8 [num_tokens] or NULL: tokens with 0 (padding) are no part
 *   of their sequence.
 *   d_seq_start int32 [Q+1], not decreasing: sequence q is tokens [start[q],
 *   start[q+1]); tokens before the first and behind the last belong to none, a
 *   sequence may be empty.  Starts outside [0, num_tokens] count as the nearer
 *   end; decreasing ones give unspecified values.  NULL: the batch is one
 *   sequence (Q == 1).
 *   An expert whose logit is NaN or -infinity has score 0; a logit of +infinity
 *   counts as the largest finite fp32.
 *   num_tokens * K below 2^31.  Scores are summed in fp32 over at most 1024
 *   tokens, then in fp64; no result depends on the order in which blocks run.
 *   d_workspace: 256-byte aligned, needs no clearing; in use by one stream (or
 *   graph in flight) at a time. */
ep_status ep_balance_loss(const ep_balance_config* cfg, const void* d_logits,
                          const int32_t* d_topk_idx, const uint8_t* d_token_mask,
                          int64_t num_tokens, const int32_t* d_seq_start, int64_t num_sequences,
                          float* d_loss, int32_t* d_counts, int32_t* d_seq_tokens,
                          float* d_score_sums, void* d_workspace, int64_t workspace_bytes,
                          void* stream);

/* Gradient of that loss with respect to the logits, the choice (so the counts)
 * held fixed: d_grad_logits [num_tokens, E], of the logits' type, written whole;
 * tokens that are masked or of no sequence get 0, as do experts without a score.
 *   d_counts, d_seq_tokens: ep_balance_loss's, or their sums over the ranks that
 *   share a batch.  d_grad_loss fp32 [1].  Logits, mask, starts and
 *   num_sequences as there. */
ep_status ep_balance_loss_backward(const ep_balance_config* cfg, const void* d_logits,
                                   const uint8_t* d_token_mask, int64_t num_tokens,
                                   const int32_t* d_seq_start, int64_t num_sequences,
                                   const int32_t* d_counts, const int32_t* d_seq_tokens,
                                   const float* d_grad_loss, void* d_grad_logits, void* stream);

/* ---- products with expert weights --------------------------------------- */

enum {
    EP_WEIGHT_BF16 = 0,    /* d_data bf16 [E, rows, cols]; cols % 8 == 0       */
    EP_WEIGHT_MXFP4 = 1,   /* OCP MX v1.0, as EP_QUANT_MXFP4: d_data two E2M1
                              codes a byte [E, rows, cols/2] (column 2i in the
                              low nibble), d_scales one E8M0 byte per 32
                              columns [E, rows, cols/32]; 255 is NaN.  An
                              element is rounded to bf16, which is exact from
                              2^-126 to the largest bf16                       */
    EP_WEIGHT_INT4 = 2,    /* d_data two codes a byte as above; an element is
                              (code - zero) * scale, with d_scales bf16
                              [E, rows, cols/group] and d_zeros uint8 of that
                              shape holding 0..15, or NULL: every zero is 8.
                              Multiplied as (16 + code) - (16 + zero): no sum of
                              a group overflows for |x| up to 2^116; an infinity
                              in x makes NaN                                   */
    EP_WEIGHT_INT8 = 3     /* for ep_matmul and ep_expert_matmul alone: d_data
                              int8 [E, rows, cols], cols % 16 == 0 and below
                              2^17; d_scales fp32 [E, rows], 4-byte aligned    */
};

/* Applied to a product's rows. */
enum {
    EP_ACT_NONE = 0,
    EP_ACT_SWIGLU = 1      /* rows = 2*I, the gate's I rows first:
                              out[i] = silu(a[i]) * a[I + i]                   */
};

/* Tokens of one ep_moe_layer call. */
#define EP_MOE_MAX_TOKENS 256

/* A stack of weight matrices, row-major, contiguous, in caller-owned device
 * memory, each 16-byte aligned (but INT8's scales). */
typedef struct ep_weights {
    int32_t format;        /* EP_WEIGHT_*                                      */
    int32_t group;         /* columns per scale: 0 (BF16, INT8), 32 (MXFP4), 32,
                              64 or 128 (INT4); divides cols                   */
    int32_t num_experts;   /* E: 1..1024                                       */
    int32_t rows;          /* M: outputs, 1..2^24                              */
    int32_t cols;          /* C: inputs, up to 2^24                            */
    int32_t reserved;      /* 0                                                */
    const void* d_data;
    const void* d_scales;  /* NULL for BF16                                    */
    const void* d_zeros;   /* INT4 only, or NULL                               */
} ep_weights;

/* y = act(x W^T) for num_rows rows and one matrix (num_experts == 1):
 *   d_x bf16 [num_rows, cols], 16-byte aligned; d_y bf16 [num_rows, M] (or
 *   [num_rows, M/2] with EP_ACT_SWIGLU), not overlapping x.  Sums in fp32, one
 *   rounding to bf16.  Made for few rows: up to 16 take one reading of the
 *   weights, more one per 16 to 32 (what LDS holds of x; ep_probe_product_path
 *   tells); num_rows * M below 2^35. */
ep_status ep_matvec(const ep_weights* w, const void* d_x, int64_t num_rows, int32_t activation,
                    void* d_y, void* stream);

/* The same for received rows: row s of an expert segment of h's layout is
 * multiplied with that expert's matrix, y[s] = act(W[e] x[s]).
 *   d_x bf16 [x_rows, cols] in receive-row order (ep_dispatch's recv_x, or an
 *   earlier product's y), d_y bf16 [x_rows, M or M/2].  Rows that hold no token
 *   (alignment padding, unfilled capacity, rows behind the last segment) are
 *   neither read nor written.  Rows at or beyond x_rows are skipped and flagged
 *   EP_FLAG_RECV_CAPACITY (ep_check_error); x_rows * M below 2^35.
 *   Made for decode batches: an expert's weights are read once per pass of its
 *   rows, and a pass holds at least the mean of rows an expert or 16, at most 16
 *   (32 where the mean is above 16).  With x so wide that LDS holds little more
 *   than the mean, experts above it are read again; a prompt's rows are right,
 *   at one reading per 16 to 32 of them.
 *   w->num_experts is the handle's; the handle has a finished layout
 *   (EP_ERR_STATE) in the expand form (EP_ERR_INVALID_ARG for non_expand, whose
 *   rows belong to ranks). */
ep_status ep_expert_matvec(const ep_handle* h, const ep_weights* w, const void* d_x,
                           int64_t x_rows, int32_t activation, void* d_y, void* stream);

/* y = act((x W^T) * x_scale * w_scale) in 8-bit integers, for num_rows rows and
 * one matrix (EP_WEIGHT_INT8, num_experts == 1):
 *   d_x int8 [num_rows, cols], 16-byte aligned, and d_x_scales fp32 [num_rows]: a
 *   dispatch's codes and scales with EP_QUANT_INT8 and quant_group = hidden, or
 *   ep_quantize_rows'; all 256 codes are values.  d_y bf16 [num_rows, M] (or
 *   [num_rows, M/2] with EP_ACT_SWIGLU), not overlapping x.
 *   Sums are exact; a sum, rounded to fp32, is multiplied by its row's scale, then
 *   by its output's, in fp32, and after the activation rounded to bf16 once.  The
 *   silu of a gate below -88.72, less than 2^-121, is -0.
 *   num_rows * M below 2^35. */
ep_status ep_matmul(const ep_weights* w, const void* d_x, const float* d_x_scales,
                    int64_t num_rows, int32_t activation, void* d_y, void* stream);

/* Bytes of device workspace with which ep_matmul_split serves a call of these
 * sizes: at most 4 MB, 0 where it does as ep_matmul. */
ep_status ep_matmul_workspace_size(const ep_weights* w, int64_t num_rows, int32_t activation,
                                   int64_t* bytes);

/* ep_matmul, to the same bits, with a workspace for the sums of products that have
 * few rows and outputs and many columns: those are split over more blocks.
 *   d_workspace: 256-byte aligned, at least ep_matmul_workspace_size bytes (NULL
 *   if that is 0), needs no clearing; in use by one stream (or graph in flight)
 *   at a time. */
ep_status ep_matmul_split(const ep_weights* w, const void* d_x, const float* d_x_scales,
                          int64_t num_rows, int32_t activation, void* d_y, void* d_workspace,
                          int64_t workspace_bytes, void* stream);

/* The same for received rows, each with its expert's matrix: rows, layout, flags
 * and states as ep_expert_matvec; the scales of rows that hold no token are not
 * read either.
 *   The kernel is chosen by the mean, num_tokens * num_topk over the experts: a
 *   mean of up to 8 rows can go to kernels that read a matrix once for each 16 of
 *   its rows (ep_probe_matmul_path tells), which costs time where a batch's tokens
 *   agree on few of many experts; the result is the same. */
ep_status ep_expert_matmul(const ep_handle* h, const ep_weights* w, const void* d_x,
                           const float* d_x_scales, int64_t x_rows, int32_t activation, void* d_y,
                           void* stream);

/* Bytes of device workspace that ep_moe_layer needs for num_tokens tokens. */
ep_status ep_moe_workspace_size(const ep_handle* h, const ep_weights* w_up,
                                const ep_weights* w_down, int64_t num_tokens, int64_t* bytes);

/* The whole expert layer of num_tokens <= EP_MOE_MAX_TOKENS tokens:
 *   a[t,k] = silu(g) * u with (g, u) = W_up[idx[t,k]] x[t]
 *   out[t] = bf16( sum over k of w[t,k] * W_down[idx[t,k]] a[t,k] )
 * with sums in fp32, a in 16 bits of mantissa (two bf16 terms) and one rounding
 * of out (ep_expert_matvec and ep_combine round a and each expert's
 * output to bf16 in between).
 *   Of h the configuration (hidden, num_topk, num_experts) and the flag word
 *   are used; its layout is neither needed nor changed, and max_tokens does not
 *   limit num_tokens.
 *   w_up: [E, 2*I, hidden], the gate's I rows first; w_down: [E, hidden, I];
 *   the formats may differ.
 *   d_x bf16 [num_tokens, hidden], 16-byte aligned; d_topk_idx int32
 *   [num_tokens, K], -1 = masked, other ids outside [0, E) are skipped and
 *   flagged EP_FLAG_BAD_EXPERT_ID; an id listed twice counts twice.
 *   d_topk_weights fp32 [num_tokens, K] or NULL (weights of 1); masked entries'
 *   weights are not used.  d_out bf16 [num_tokens, hidden]: a token without an
 *   expert gets +0.  d_out may be d_x.
 *   d_workspace: 256-byte aligned, at least ep_moe_workspace_size bytes, needs
 *   no clearing; in use by one stream (or graph in flight) at a time.
 *   Two kernels for up to 16 tokens and 32 entries of topk_idx (8 with w_down in
 *   INT4 groups of 32 or 64) whose activations fit 64 KB of LDS, 2 * entries *
 *   (2 * I' + 16) bytes with I' = I rounded up to a multiple of 64 (bf16 w_down)
 *   or 256 (4 bits); else three.  The result does not depend on the order in
 *   which blocks run. */
ep_status ep_moe_layer(const ep_handle* h, const ep_weights* w_up, const ep_weights* w_down,
                       const void* d_x, const int32_t* d_topk_idx, const float* d_topk_weights,
                       int64_t num_tokens, void* d_out, void* d_workspace, int64_t workspace_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif
