/*
 * mmq_layer.h -- C ABI of the layer operators of libmmq.so, beside the q4_K x q8_1 product of
 * mmq.h: the product with an epilogue, its gated two-matrix form, a mixture-of-experts layer for a
 * few tokens with its router, and the layer's products grouped by expert for any number of tokens.
 *
 * P below is the product of mmq.h, P_ij = sum_b (da_ib dsv_jb S_ijb + dmv_jb da_ib sa_ib), over
 * activations quantized to q8_1 and q4_K weights; everything after it is float32.
 *
 * The conventions of mmq.h hold: DEVICE pointers owned by the caller, 16-byte aligned, not
 * overlapping unless an entry point says so; `stream` is a hipStream_t; every argument is
 * validated on the host before anything is launched; nothing is allocated and nothing
 * synchronizes, so every call can be captured into a HIP graph; results are deterministic; return
 * values are mmq_status codes; mmq_last_error reports the calling thread's last error. Scratch
 * and workspaces belong to one call at a time: calls (or replayed graphs) that share one must not
 * overlap.
 */
#ifndef MMQ_LAYER_H
#define MMQ_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "mmq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations: silu(v) = v / (1 + e^-v); gelu(v) = v/2 (1 + erf(v / sqrt 2)); gelu_tanh(v) =
 * v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))); relu passes NaN. */
enum mmq_act {
  MMQ_ACT_NONE = 0,
  MMQ_ACT_RELU = 1,
  MMQ_ACT_SILU = 2,
  MMQ_ACT_GELU = 3,
  MMQ_ACT_GELU_TANH = 4
};

/* ---------------------------------------------------------------- the product's epilogue */

typedef struct mmq_epilogue {
  const float* bias;     /* [N], added before the activation, or NULL */
  const float* residual; /* [M][N], added after it, or NULL; may be C itself */
  int32_t act;           /* enum mmq_act */
  int32_t reserved;      /* must be 0 */
} mmq_epilogue;

/*
 * mmq_q4K_q8_1_epilogue: C[M][N] = act(P + bias) + residual, in the product's own kernels (every
 * tile of mmq_q4K_q8_1_ex; with split-K in the kernel that adds the partial planes). epi == NULL
 * or an empty one is mmq_q4K_q8_1_ex, bit for bit; otherwise P is, bit for bit, what that call
 * computes with the same tile and splits (mmq_last_kernel reports them; with a workspace the guard
 * counts the second kernel of a split as well, so that it may leave K whole where the plain
 * product's, which mmq_plan answers for, splits it). Same limits, options and errors; MMQ_E_ARG for a
 * bad epilogue (an act that is none, a misaligned bias or residual, reserved != 0). bias and residual
 * may not overlap C, except a residual that is C.
 */
int mmq_q4K_q8_1_epilogue(int64_t M, int64_t N, int64_t K, const void* q8, const void* w_rep,
                          float* C, void* stream, const mmq_epilogue* epi,
                          const mmq_options* opt);

/* As mmq_q4K_f32 (few tokens, 1 <= M <= 128, float32 activations quantized in the product, one
 * launch) with the epilogue. Against quantize_q8_1 and the product (graph replays, residual): 1
 * token 5.0 / 7.1 us at 4096 x 4096, 13.6 / 15.4 at 22016 x 4096; 2 tokens 6.0 / 7.5 and 18.3 / 16.1;
 * 4 tokens 7.9 / 8.4 and 38 / 20. */
int mmq_q4K_f32_epilogue(int64_t M, int64_t N, int64_t K, const float* x, const void* w_rep,
                         float* C, void* stream, const mmq_epilogue* epi);

/* ---------------------------------------------------------------- the gated product */

/*
 * The first half of a gated feed-forward: H[M][F] = act(X Wg^T) * (X Wu^T), both matrices F x K
 * q4_K. They are repacked together, 8 rows of one and 8 of the other in turn, so that one pass
 * over the activations and one kernel form both products and nothing but H is written.
 *
 * mmq_q4K_pair_bytes: ceil(F/16) * (K/256) * 4608, the size of a repacked pair. K % 256 == 0,
 * F <= 2^29.
 * repack_q4_K_pair: the records of repack_q4_K over the packed rows: packed row 16 b + r is row
 * 8 b + r of w_gate for r < 8, row 8 b + r - 8 of w_up for r >= 8; rows past F are zero, up to a
 * multiple of 32 packed rows. Run once per pair; ceil(F/16) * (K/256) < 2^24. Errors as repack_q4_K.
 */
int mmq_q4K_pair_bytes(int64_t F, int64_t K, size_t* bytes);
int repack_q4_K_pair(const void* w_gate, const void* w_up, int64_t F, int64_t K, void* w_pair,
                     void* stream);

/* Bytes of split-K workspace mmq_q4K_q8_1_gated would use, given an unlimited one. Host only. */
int mmq_gated_workspace_bytes(int64_t M, int64_t F, int64_t K, size_t* bytes);

/*
 * mmq_q4K_q8_1_gated: q8 from quantize_q8_1 (M x K), w_pair from repack_q4_K_pair (F, K); H
 * overwritten. Each of the two sums is what mmq_q4K_q8_1_ex computes for the packed matrix of
 * 32 * ceil(F/16) rows, whose kernels, options and limits these are (mmq_last_kernel reports that
 * product; the guard's choice is mmq_q4K_q8_1_epilogue's). MMQ_ACT_NONE gives the bilinear form.
 * mmq_q4K_f32_gated: few tokens (M <= 128) from float32 activations, as mmq_q4K_f32.
 */
int mmq_q4K_q8_1_gated(int64_t M, int64_t F, int64_t K, const void* q8, const void* w_pair,
                       float* H, void* stream, int32_t act, const mmq_options* opt);
int mmq_q4K_f32_gated(int64_t M, int64_t F, int64_t K, const float* x, const void* w_pair,
                      float* H, void* stream, int32_t act);

/* ---------------------------------------------------------------- mixture of experts */

/* Limits of a plan and of the products that read it (the router alone takes up to 2^25 tokens). */
#define MMQ_MOE_MAX_TOKENS 64
#define MMQ_MOE_MAX_PAIRS 512   /* M * k */
#define MMQ_MOE_MAX_EXPERTS 512
#define MMQ_MOE_MAX_SLOTS 64    /* k, and k <= E */

enum mmq_score {
  MMQ_SCORE_SOFTMAX = 0, /* over all E experts */
  MMQ_SCORE_SIGMOID = 1  /* of each logit by itself */
};

/* Bytes of a plan for M tokens, E experts, k slots each: 4 * (4 + 4 * min(E, M*k) + M*k). */
int mmq_moe_plan_bytes(int64_t M, int64_t E, int64_t k, size_t* bytes);

/*
 * mmq_moe_plan: the plan of the experts' products from ids (int32 [M][k], the expert of each
 * (token, slot) pair p = t * k + s). An id outside [0, E) names no expert: its slot contributes
 * nothing (a padded token, an expert of another device). A token may name an expert twice. The
 * plan, int32: [used experts, pairs with an expert, 0, 0]; then min(E, M*k) entries [expert,
 * first, pairs, 0], the used experts in increasing order, then [-1, 0, 0, 0]; then the M*k pairs
 * sorted by expert, pairs of one expert in increasing order, those without one replaced by -1 at
 * the end. `first` counts from the first pair. The products bound-check what they read of a plan;
 * a plan made for other M, E, k gives unspecified results.
 */
int mmq_moe_plan(int64_t M, int64_t E, int64_t k, const int32_t* ids, int32_t* plan,
                 void* stream);

/*
 * mmq_moe_route: per token t the k experts of the greatest logits[t][0..E), in decreasing order,
 * equal logits in increasing order of expert, into ids[t][0..k), and their weights:
 *   MMQ_SCORE_SOFTMAX  e^(l_s - max) / sum over all E experts, or over the k chosen with renorm
 *   MMQ_SCORE_SIGMOID  1 / (1 + e^-l_s), divided by the sum over the k chosen with renorm: by the
 *                      scores' ratios, however small they are, as long as the greatest of them is
 *                      not 0 in float32 (a logit below -150 ln 2 = -103.97); then all weigh 0
 * A logit of -inf or NaN is never chosen and weighs nothing (a masked expert); a token with fewer
 * than k others gets id -1 and weight 0 in the slots that are left. Where the greatest logit is
 * +inf, the experts that have it share the softmax. plan may be NULL (then 1 <= M <= 2^25);
 * otherwise it is written as mmq_moe_plan would.
 * 1 <= E <= 512, 1 <= k <= min(E, 64).
 */
int mmq_moe_route(int64_t M, int64_t E, int64_t k, const float* logits, int32_t score,
                  int32_t renorm, int32_t* ids, float* weights, int32_t* plan, void* stream);

/*
 * mmq_q4K_moe_gated: H[p][F] = act(x[t] Wg(e)^T) * (x[t] Wu(e)^T) for every pair p = t*k + s of
 * the plan with an expert e; rows of H of pairs without one are left as they were. x float32
 * [M][D]; w_pairs: E repacked pairs (F, D) one behind the other; q8: scratch of
 * mmq_q8_1_bytes(M, D) bytes (not written for one token, whose values the product quantizes
 * itself). A used expert's weights are read once per 16 of its pairs (for one token: once per pair).
 * M <= 64, M*k <= 512, E <= 512, D % 256 == 0, D <= 2^24, min(E, M*k) * ceil(F/16) < 2^23.
 * Errors: MMQ_E_ARG, MMQ_E_SHAPE, MMQ_E_LDS, MMQ_E_DEVICE, MMQ_E_HIP.
 */
int mmq_q4K_moe_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, const float* x,
                      const int32_t* plan, const void* w_pairs, float* H, void* q8, int32_t act,
                      void* stream);

/*
 * mmq_q4K_moe_down: out[t][D] = residual[t] + sum over the slots s of weights[t][s] * (H[p] W(e)^T)
 * over the plan's pairs p = t*k + s; slots without an expert add nothing, and a token without any
 * gets its residual (0 if residual is NULL). H float32 [M*k][F] (rows of pairs without an expert
 * are not used); weights float32 [M][k]; w_down: E repacked q4_K matrices (D, F) one behind the
 * other; q8: scratch of mmq_q8_1_bytes(M*k, F) bytes, as above; residual may be out itself. A used
 * expert's weights are read once per 3 to 16 of its pairs (one token: per pair), the number chosen
 * from M, E, k and D as if the experts were named evenly: a call whose tokens agree on one expert of
 * many takes up to 2.2 times as long as one whose tokens do not.
 * M <= 64, M*k <= 512, E <= 512, F % 256 == 0, F <= 2^24, M*k*F < 2^31, D <= 2^25. Errors as
 * mmq_q4K_moe_gated.
 */
int mmq_q4K_moe_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* H,
                     const int32_t* plan, const float* weights, const void* w_down,
                     const float* residual, float* out, void* q8, void* stream);

/*
 * mmq_q4K_moe: the whole layer for a few tokens: mmq_moe_route, mmq_q4K_moe_gated and
 * mmq_q4K_moe_down on the router's logits [M][E], bit for bit what those calls give one after the
 * other. workspace: mmq_moe_workspace_bytes(M, E, k, D, F) bytes (D, F multiples of 256).
 */
int mmq_moe_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, size_t* bytes);
int mmq_q4K_moe(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* x,
                const float* logits, int32_t score, int32_t renorm, const void* w_pairs,
                int32_t act, const void* w_down, const float* residual, float* out,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- products grouped by expert */

/*
 * The mixture-of-experts layer for more tokens than a plan takes, and for any raggedness: the
 * (token, slot) pairs p = t*k + s are sorted by expert on the device, and one launch runs each
 * expert's rows, however many, against its matrix. Nothing about the counts has to be known on the
 * host. Per pair the products are mmq_q4K_q8_1's for its row and its expert's matrix, within the same
 * bound; the order in which K is added up depends on M, E, k, N and K (and the device's compute units),
 * not on the ids.
 *
 * Limits of all of them: 1 <= M*k <= 2^21, E <= 512, k <= min(E, 64).
 */
#define MMQ_GROUP_MAX_PAIRS (1 << 21)

/*
 * mmq_moe_group: the groups of ids (int32 [M][k], the expert of each pair, from mmq_moe_route or
 * elsewhere; an id outside [0, E) names no expert: a padded token, an expert of another device).
 * groups, int32, mmq_moe_group_bytes(M, E, k) bytes, each part starting at a multiple of 4 words:
 *   offsets[E + 1]  the pairs of expert e are order[offsets[e] .. offsets[e + 1])
 *   order[M*k]      the pairs sorted by expert, those of one expert in increasing order, those without
 *                   one replaced by -1 at the end
 *   place[M*k]      where each pair is in order, -1 without an expert
 * and behind them words of its own (unspecified). The products bound-check what they read of the
 * groups; groups made for other M, E, k give unspecified results.
 */
int mmq_moe_group_bytes(int64_t M, int64_t E, int64_t k, size_t* bytes);
int mmq_moe_group(int64_t M, int64_t E, int64_t k, const int32_t* ids, int32_t* groups,
                  void* stream);

/*
 * mmq_q4K_grouped: C[p][N] = act(x[r] W(e)^T) for every pair p with an expert e; rows of C of pairs
 * without one are left as they were. per_pair = 0: x float32 [M][K], a row per token, r = p / k;
 * per_pair = 1: x [M*k][K], a row per pair, r = p. w_rep: E repacked q4_K matrices (N, K) one behind
 * the other; q8: scratch of mmq_q8_1_bytes(rows of x, K) bytes (in a layout of its own).
 * mmq_q4K_grouped_gated: H[p][F] = act(x[p / k] Wg(e)^T) * (x[p / k] Wu(e)^T), x float32 [M][D],
 * w_pairs: E repacked pairs (F, D); q8: scratch of mmq_q8_1_bytes(M, D) bytes.
 * mmq_q4K_moe_gated and _down take up to 64 tokens with a plan; they are the faster ones for few tokens
 * (gated and down of 8 tokens, 8 of 64 experts, D = 2048, F = 1024: 28 and 16 us against 30 and 24; 2 of
 * 8, 4096, 11008: 85 and 43 against 100 and 49), and where an expert gets some 4 to 8 of the pairs on
 * average the two meet (64 tokens: 45 and 37 against 39 and 29; 128 and 76 against 109 and 54).
 * K % 256 == 0, K <= 2^24, (rows of x)*K < 2^31, N <= 2^30, and (M*k/32 + min(E, M*k)) * ceil(N/256)
 * < 2^23 - 4096 (gated: of its 32 * ceil(F/16) packed rows).
 * Errors: MMQ_E_ARG, MMQ_E_SHAPE, MMQ_E_LDS, MMQ_E_DEVICE, MMQ_E_HIP.
 */
int mmq_q4K_grouped(int64_t M, int64_t E, int64_t k, int64_t N, int64_t K, const float* x,
                    int32_t per_pair, const int32_t* groups, const void* w_rep, float* C, void* q8,
                    int32_t act, void* stream);
int mmq_q4K_grouped_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, const float* x,
                          const int32_t* groups, const void* w_pairs, float* H, void* q8,
                          int32_t act, void* stream);

/*
 * mmq_q4K_grouped_down: out[t][D] = residual[t] + sum over the slots s of weights[t][s] * (H[p]
 * W(e)^T) over the pairs p = t*k + s with an expert, in float32 and in the order of the slots; a token
 * without any gets its residual (0 if residual is NULL). H float32 [M*k][F] (rows of pairs without
 * an expert may hold anything: they are read, not used); weights float32 [M][k]; w_down: E repacked
 * q4_K matrices (D, F); residual may be out itself. workspace:
 * mmq_grouped_down_workspace_bytes(M, E, k, D, F) bytes, for H in q8_1 and the pairs' products.
 * Limits as mmq_q4K_grouped with N = D, K = F and M*k rows; M * ceil(D/256) < 2^24.
 */
int mmq_grouped_down_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F,
                                     size_t* bytes);
int mmq_q4K_grouped_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* H,
                         const int32_t* groups, const float* weights, const void* w_down,
                         const float* residual, float* out, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * mmq_q4K_grouped_moe: the whole layer: mmq_moe_route on the router's logits [M][E], mmq_moe_group,
 * mmq_q4K_grouped_gated and mmq_q4K_grouped_down, bit for bit what those calls give one after the
 * other. workspace: mmq_grouped_moe_workspace_bytes(M, E, k, D, F) bytes (D, F multiples of 256).
 */
int mmq_grouped_moe_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F,
                                    size_t* bytes);
int mmq_q4K_grouped_moe(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* x,
                        const float* logits, int32_t score, int32_t renorm, const void* w_pairs,
                        int32_t act, const void* w_down, const float* residual, float* out,
                        void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MMQ_LAYER_H */
