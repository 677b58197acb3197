// Host side of the products grouped by expert (include/mmq_layer.h): argument checks, workspaces and
// launches. As in api.cpp nothing touches the device before every argument has been checked.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "grouped_internal.h"
#include "mmq.h"
#include "mmq_layer.h"
#include "moe_internal.h"

namespace {

using mmq::check_pointers;
using mmq::fail;
using mmq::GroupedShape;
using mmq::GroupLayout;
using mmq::hip_status;

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 24;
static_assert(MMQ_GROUP_MAX_PAIRS == mmq::kGroupMaxPairs, "limits");
static_assert(MMQ_MOE_MAX_EXPERTS == mmq::kGroupMaxExperts, "limits");

int check_groups(int64_t M, int64_t E, int64_t k) {
  if (M <= 0 || E <= 0 || k <= 0)
    return fail(MMQ_E_ARG, "M, E, k must be positive (%lld, %lld, %lld)", (long long)M,
                (long long)E, (long long)k);
  if (E > mmq::kGroupMaxExperts) return fail(MMQ_E_SHAPE, "E = %lld is above 512", (long long)E);
  if (k > E || k > MMQ_MOE_MAX_SLOTS)
    return fail(MMQ_E_SHAPE, "k = %lld is above min(E, %d)", (long long)k, MMQ_MOE_MAX_SLOTS);
  if (M > mmq::kGroupMaxPairs / k)
    return fail(MMQ_E_SHAPE, "M*k is above 2^21 pairs (M = %lld, k = %lld)", (long long)M,
                (long long)k);
  return MMQ_OK;
}

// One product over E matrices of `rows` weight rows (of which N are packed) x K, q_rows token rows.
int check_product(int64_t M, int64_t E, int64_t k, const char* rows_name, int64_t rows,
                  bool gated, const char* k_name, int64_t K, int64_t q_rows) {
  if (rows <= 0 || K <= 0)
    return fail(MMQ_E_ARG, "%s and %s must be positive (%lld, %lld)", rows_name, k_name,
                (long long)rows, (long long)K);
  if (K % MMQ_QK_K)
    return fail(MMQ_E_SHAPE, "%s = %lld is not a multiple of 256", k_name, (long long)K);
  if (rows > (gated ? kMaxDim / 2 : kMaxDim) || K > kMaxK)
    return fail(MMQ_E_SHAPE, "%s = %lld or %s = %lld too large", rows_name, (long long)rows, k_name,
                (long long)K);
  if (q_rows * K >= ((int64_t)1 << 31))
    return fail(MMQ_E_SHAPE, "activations of %lld x %lld: 2^31 values or more", (long long)q_rows,
                (long long)K);
  const int64_t N = gated ? mmq::pair_rows(rows) : rows;
  // Workgroups of 256 work-items on 32 x 128 tiles or 512 on 128 x 256: below 2^32 work-items, with a
  // round of them more (grouped.hip; the split forms' grids are smaller, grouped_form).
  const int64_t P = M * k, tiles = P / 32 + (E < P ? E : P);
  if (tiles * ((N + 255) / 256) >= ((int64_t)1 << 23) - 4096)
    return fail(MMQ_E_SHAPE, "M*k = %lld, E = %lld, %s = %lld: 2^23 - 4096 tiles or more",
                (long long)P, (long long)E, rows_name, (long long)rows);
  return MMQ_OK;
}

int check_act(int32_t act) {
  return act < MMQ_ACT_NONE || act > MMQ_ACT_GELU_TANH
             ? fail(MMQ_E_ARG, "act %d is not an mmq_act", act)
             : MMQ_OK;
}

// The device's compute units, and that the product's kernel fits its LDS.
int check_device(const GroupedShape& g, int64_t* cus) {
  int64_t budget = 0;
  const int st = mmq::api_current_device(&budget, cus);
  if (st) return st;
  const int64_t need = mmq::grouped_lds_bytes(mmq::grouped_form(g, *cus));
  if (need > budget)
    return fail(MMQ_E_LDS, "the grouped product needs %lld bytes of LDS, the device allows %lld",
                (long long)need, (long long)budget);
  return MMQ_OK;
}

GroupedShape gated_shape(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D) {
  return GroupedShape{M * k, E, mmq::pair_rows(F), D, M, k};
}
GroupedShape down_shape(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F) {
  return GroupedShape{M * k, E, D, F, M * k, 1};
}

int check_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, int32_t act) {
  int st = check_groups(M, E, k);
  if (!st) st = check_product(M, E, k, "F", F, true, "D", D, M);
  return st ? st : check_act(act);
}
int check_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F) {
  int st = check_groups(M, E, k);
  if (!st) st = check_product(M, E, k, "D", D, false, "F", F, M * k);
  if (!st && (D + 255) / 256 * M >= ((int64_t)1 << 24))
    st = fail(MMQ_E_SHAPE, "M * ceil(D/256) is not below 2^24 (M = %lld, D = %lld)", (long long)M,
              (long long)D);
  return st;
}

// Workspaces, each part at a 256-byte boundary.
struct Taker {
  int64_t at = 0;
  int64_t operator()(int64_t n) {
    const int64_t here = at;
    at = mmq::round256(at + n);
    return here;
  }
};
struct DownSpace {
  int64_t q8, Y, total;
};
DownSpace down_space(int64_t M, int64_t k, int64_t D, int64_t F) {
  Taker take;
  DownSpace w;
  w.q8 = take(mmq::q8_total_bytes(M * k, F));
  w.Y = take(4 * M * k * D);
  w.total = take.at;
  return w;
}
// The layer: x is quantized into the place that H's q8_1 form has after it.
struct LayerSpace {
  int64_t ids, weights, groups, H, down, total;
};
LayerSpace layer_space(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F) {
  Taker take;
  LayerSpace w;
  w.ids = take(4 * M * k);
  w.weights = take(4 * M * k);
  w.groups = take(4 * GroupLayout{M * k, E}.words());
  w.H = take(4 * M * k * F);
  const int64_t qx = mmq::q8_total_bytes(M, D), down = down_space(M, k, D, F).total;
  w.down = take(qx > down ? qx : down);
  w.total = take.at;
  return w;
}

hipError_t run_product(const GroupedShape& g, const float* x, const int32_t* groups, const void* w,
                       float* out, void* q8, const mmq::Epilogue& epi, int64_t cus,
                       hipStream_t s) {
  const hipError_t e = mmq::launch_quantize_rows(x, g.q_rows, g.K, q8, s);
  return e != hipSuccess ? e : mmq::launch_grouped(q8, groups, w, out, g, epi, cus, s);
}

hipError_t run_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, const float* x,
                     const int32_t* groups, const void* w, float* H, void* q8, int32_t act,
                     int64_t cus, hipStream_t s) {
  mmq::Epilogue epi;
  epi.kind = mmq::kEpiGated;
  epi.act = act;
  epi.F = F;
  return run_product(gated_shape(M, E, k, F, D), x, groups, w, H, q8, epi, cus, s);
}

hipError_t run_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* H,
                    const int32_t* groups, const float* weights, const void* w,
                    const float* residual, float* out, void* workspace, int64_t cus, hipStream_t s) {
  const DownSpace sp = down_space(M, k, D, F);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* Y = reinterpret_cast<float*>(ws + sp.Y);
  mmq::Epilogue epi;
  epi.kind = mmq::kEpiAct;
  const hipError_t e = run_product(down_shape(M, E, k, D, F), H, groups, w, Y, ws + sp.q8, epi, cus, s);
  if (e != hipSuccess) return e;
  return mmq::launch_combine(Y, groups + GroupLayout{M * k, E}.place(), weights, residual, out, M, k,
                             D, s);
}

int check_bytes(size_t have, int64_t need) {
  return have < (size_t)need
             ? fail(MMQ_E_ARG, "the call needs %lld bytes of workspace, %llu given",
                    (long long)need, (unsigned long long)have)
             : MMQ_OK;
}

}  // namespace

extern "C" {

int mmq_moe_group_bytes(int64_t M, int64_t E, int64_t k, size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  const int st = check_groups(M, E, k);
  if (st) return st;
  *bytes = (size_t)(4 * GroupLayout{M * k, E}.words());
  return mmq::api_ok();
}

int mmq_moe_group(int64_t M, int64_t E, int64_t k, const int32_t* ids, int32_t* groups,
                  void* stream) {
  int st = check_groups(M, E, k);
  if (!st) st = check_pointers({ids, groups});
  if (!st) st = mmq::api_current_device();
  if (st) return st;
  return hip_status("mmq_moe_group",
                    mmq::launch_group(ids, M * k, E, groups, static_cast<hipStream_t>(stream)));
}

int mmq_q4K_grouped(int64_t M, int64_t E, int64_t k, int64_t N, int64_t K, const float* x,
                    int32_t per_pair, const int32_t* groups, const void* w_rep, float* C, void* q8,
                    int32_t act, void* stream) {
  int st = check_groups(M, E, k);
  if (!st && per_pair != 0 && per_pair != 1) st = fail(MMQ_E_ARG, "per_pair must be 0 or 1");
  const int64_t rows = !st && per_pair ? M * k : M;
  if (!st) st = check_product(M, E, k, "N", N, false, "K", K, rows);
  if (!st) st = check_act(act);
  if (!st) st = check_pointers({x, groups, w_rep, C, q8});
  if (st) return st;
  const GroupedShape g{M * k, E, N, K, rows, per_pair ? 1 : k};
  int64_t cus = 0;
  if ((st = check_device(g, &cus))) return st;
  mmq::Epilogue epi;
  epi.kind = mmq::kEpiAct;
  epi.act = act;
  return hip_status("mmq_q4K_grouped", run_product(g, x, groups, w_rep, C, q8, epi, cus,
                                                   static_cast<hipStream_t>(stream)));
}

int mmq_q4K_grouped_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, const float* x,
                          const int32_t* groups, const void* w_pairs, float* H, void* q8,
                          int32_t act, void* stream) {
  int st = check_gated(M, E, k, F, D, act);
  if (!st) st = check_pointers({x, groups, w_pairs, H, q8});
  int64_t cus = 0;
  if (!st) st = check_device(gated_shape(M, E, k, F, D), &cus);
  if (st) return st;
  return hip_status("mmq_q4K_grouped_gated",
                    run_gated(M, E, k, F, D, x, groups, w_pairs, H, q8, act, cus,
                              static_cast<hipStream_t>(stream)));
}

int mmq_grouped_down_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F,
                                     size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  const int st = check_down(M, E, k, D, F);
  if (st) return st;
  *bytes = (size_t)down_space(M, k, D, F).total;
  return mmq::api_ok();
}

int mmq_q4K_grouped_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* H,
                         const int32_t* groups, const float* weights, const void* w_down,
                         const float* residual, float* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int st = check_down(M, E, k, D, F);
  if (!st) st = check_pointers({H, groups, weights, w_down, out, workspace}, residual);
  if (!st) st = check_bytes(workspace_bytes, down_space(M, k, D, F).total);
  int64_t cus = 0;
  if (!st) st = check_device(down_shape(M, E, k, D, F), &cus);
  if (st) return st;
  return hip_status("mmq_q4K_grouped_down",
                    run_down(M, E, k, D, F, H, groups, weights, w_down, residual, out, workspace, cus,
                             static_cast<hipStream_t>(stream)));
}

int mmq_grouped_moe_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F,
                                    size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  int st = check_gated(M, E, k, F, D, MMQ_ACT_NONE);
  if (!st) st = check_down(M, E, k, D, F);
  if (st) return st;
  *bytes = (size_t)layer_space(M, E, k, D, F).total;
  return mmq::api_ok();
}

int mmq_q4K_grouped_moe(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* x,
                        const float* logits, int32_t score, int32_t renorm, const void* w_pairs,
                        int32_t act, const void* w_down, const float* residual, float* out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gated(M, E, k, F, D, act);
  if (!st) st = check_down(M, E, k, D, F);
  if (!st && score != MMQ_SCORE_SOFTMAX && score != MMQ_SCORE_SIGMOID)
    st = fail(MMQ_E_ARG, "score %d is not an mmq_score", score);
  if (!st && renorm != 0 && renorm != 1) st = fail(MMQ_E_ARG, "renorm must be 0 or 1");
  if (!st) st = check_pointers({x, logits, w_pairs, w_down, out, workspace}, residual);
  if (st) return st;
  const LayerSpace w = layer_space(M, E, k, D, F);
  if ((st = check_bytes(workspace_bytes, w.total))) return st;
  int64_t cus = 0;
  if ((st = check_device(gated_shape(M, E, k, F, D), &cus))) return st;
  if ((st = check_device(down_shape(M, E, k, D, F), &cus))) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* ids = reinterpret_cast<int*>(ws + w.ids);
  float* weights = reinterpret_cast<float*>(ws + w.weights);
  int* groups = reinterpret_cast<int*>(ws + w.groups);
  float* H = reinterpret_cast<float*>(ws + w.H);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = mmq::launch_moe_route(logits, M, E, k, score, renorm, ids, weights, nullptr, s);
  if (e == hipSuccess) e = mmq::launch_group(ids, M * k, E, groups, s);
  if (e == hipSuccess) e = run_gated(M, E, k, F, D, x, groups, w_pairs, H, ws + w.down, act, cus, s);
  if (e == hipSuccess)
    e = run_down(M, E, k, D, F, H, groups, weights, w_down, residual, out, ws + w.down, cus, s);
  return hip_status("mmq_q4K_grouped_moe", e);
}

}  // extern "C"
