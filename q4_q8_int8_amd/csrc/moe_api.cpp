// Host side of the mixture-of-experts entry points of include/mmq_layer.h: argument checks, the
// layer's workspace, and the launches. As in api.cpp nothing touches the device before every
// argument has been checked.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "mmq.h"
#include "mmq_internal.h"
#include "mmq_layer.h"
#include "moe_internal.h"

namespace {

int fail(int status, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return mmq::api_fail(status, msg);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t)1 << 30;
// A grid holds fewer than 2^32 work-items: the router launches 64 per token, the down product at most
// 64 per output column (1024 per 16 columns; with 8, as many workgroups as compute units).
constexpr int64_t kMaxRouted = (int64_t)1 << 25, kMaxDown = (int64_t)1 << 25;
constexpr int64_t kMaxK = (int64_t)1 << 24;
constexpr int64_t kMaxSlots = MMQ_MOE_MAX_SLOTS;
static_assert(MMQ_MOE_MAX_TOKENS == mmq::kMoeMaxTokens, "limits");
static_assert(MMQ_MOE_MAX_PAIRS == mmq::kMoeMaxPairs, "limits");
static_assert(MMQ_MOE_MAX_EXPERTS == mmq::kMoeMaxExperts, "limits");

// Tokens, experts and slots of the router; with `planned` within a plan's limits too.
int check_routing(int64_t M, int64_t E, int64_t k, bool planned) {
  if (M <= 0 || E <= 0 || k <= 0)
    return fail(MMQ_E_ARG, "M, E, k must be positive (%lld, %lld, %lld)", (long long)M,
                (long long)E, (long long)k);
  if (E > mmq::kMoeMaxExperts) return fail(MMQ_E_SHAPE, "E = %lld is above 512", (long long)E);
  if (k > E || k > kMaxSlots)
    return fail(MMQ_E_SHAPE, "k = %lld is above min(E, %lld)", (long long)k, (long long)kMaxSlots);
  if (M > kMaxRouted) return fail(MMQ_E_SHAPE, "M above 2^25");
  if (planned && (M > mmq::kMoeMaxTokens || M * k > mmq::kMoeMaxPairs))
    return fail(MMQ_E_SHAPE, "a plan is for few tokens: M <= 64 and M*k <= 512 (%lld, %lld)",
                (long long)M, (long long)(M * k));
  return MMQ_OK;
}

// One product over E matrices of rows x K weights, from a q8 buffer of q8_rows x K.
int check_product(const char* rows_name, int64_t rows, const char* k_name, int64_t K,
                  int64_t q8_rows, int64_t max_rows) {
  if (rows <= 0 || K <= 0)
    return fail(MMQ_E_ARG, "%s and %s must be positive (%lld, %lld)", rows_name, k_name,
                (long long)rows, (long long)K);
  if (K % MMQ_QK_K) return fail(MMQ_E_SHAPE, "%s = %lld is not a multiple of 256", k_name, (long long)K);
  if (rows > max_rows || K > kMaxK)
    return fail(MMQ_E_SHAPE, "%s = %lld or %s = %lld too large", rows_name, (long long)rows, k_name,
                (long long)K);
  if (q8_rows * K >= ((int64_t)1 << 31))
    return fail(MMQ_E_SHAPE, "activations of %lld x %lld: 2^31 values or more", (long long)q8_rows,
                (long long)K);
  return MMQ_OK;
}

int check_pointers(std::initializer_list<const void*> needed, const void* optional = nullptr) {
  for (const void* p : needed) {
    if (!p) return fail(MMQ_E_ARG, "null device pointer");
    if (!aligned16(p)) return fail(MMQ_E_ARG, "device pointers must be 16-byte aligned");
  }
  if (!aligned16(optional)) return fail(MMQ_E_ARG, "device pointers must be 16-byte aligned");
  return MMQ_OK;
}

int hip_status(const char* what, hipError_t e) {
  return e == hipSuccess ? mmq::api_ok()
                         : fail(MMQ_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

// The device's compute units, and that the down product's kernel fits its LDS (the gated ones and
// the router use less than the 64 KiB that every kernel may).
int check_device(const mmq::MoeShape& m, int64_t* compute_units) {
  int64_t budget = 0;
  const int st = mmq::api_current_device(&budget, compute_units);
  if (st) return st;
  const int64_t need = mmq::moe_down_lds_bytes(m, *compute_units);
  if (need > budget)
    return fail(MMQ_E_LDS, "the experts' down product needs %lld bytes of LDS, the device allows "
                           "%lld", (long long)need, (long long)budget);
  return MMQ_OK;
}

int check_act(int32_t act) {
  return act < MMQ_ACT_NONE || act > MMQ_ACT_GELU_TANH
             ? fail(MMQ_E_ARG, "act %d is not an mmq_act", act)
             : MMQ_OK;
}

int check_route_options(int32_t score, int32_t renorm) {
  if (score != MMQ_SCORE_SOFTMAX && score != MMQ_SCORE_SIGMOID)
    return fail(MMQ_E_ARG, "score %d is not an mmq_score", score);
  if (renorm != 0 && renorm != 1) return fail(MMQ_E_ARG, "renorm must be 0 or 1");
  return MMQ_OK;
}

int check_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, int32_t act) {
  int st = check_routing(M, E, k, true);
  if (!st) st = check_product("F", F, "D", D, M, kMaxDim);
  if (!st) st = check_act(act);
  // at most two workgroups of 256 work-items per (expert, 16 columns), on a 1-D grid of fewer than
  // 2^32 work-items
  const int64_t entries = mmq::MoeShape{M, E, k, D, F}.entries();
  if (!st && (F + 15) / 16 * entries >= ((int64_t)1 << 23))
    st = fail(MMQ_E_SHAPE, "min(E, M*k) * ceil(F/16) = %lld is not below 2^23",
              (long long)((F + 15) / 16 * entries));
  return st;
}

int check_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F) {
  const int st = check_routing(M, E, k, true);
  return st ? st : check_product("D", D, "F", F, M * k, kMaxDown);
}

// The layer's workspace: each part at a 256-byte boundary. H is quantized into `q8`, which x used
// before it.
struct Workspace {
  int64_t ids, weights, plan, H, q8, total;
};
Workspace layout(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F) {
  Workspace w;
  int64_t at = 0;
  auto take = [&at](int64_t n) {
    const int64_t here = at;
    at = mmq::round256(at + n);
    return here;
  };
  const mmq::MoeShape m{M, E, k, D, F};
  w.ids = take(4 * m.pairs());
  w.weights = take(4 * m.pairs());
  w.plan = take(4 * (mmq::kPlanHead + 4 * m.entries() + m.pairs()));
  w.H = take(4 * m.pairs() * F);
  const int64_t qx = mmq::q8_total_bytes(M, D), qh = mmq::q8_total_bytes(m.pairs(), F);
  w.q8 = take(qx > qh ? qx : qh);
  w.total = at;
  return w;
}

hipError_t run_gated(const mmq::MoeShape& m, const float* x, const int32_t* plan, const void* w,
                     float* H, void* q8, int32_t act, hipStream_t s) {
  if (mmq::moe_fused(m.M)) return mmq::launch_moe_gated(x, plan, w, H, m, act, s);
  const hipError_t e = mmq::launch_quantize_q8_1(x, m.M, m.D, q8, s);
  return e != hipSuccess ? e : mmq::launch_moe_gated(q8, plan, w, H, m, act, s);
}

hipError_t run_down(const mmq::MoeShape& m, const float* H, const int32_t* plan,
                    const float* weights, const void* w, const float* residual, float* out,
                    void* q8, int64_t cus, hipStream_t s) {
  if (mmq::moe_fused(m.M))
    return mmq::launch_moe_down(H, plan, weights, w, residual, out, m, cus, s);
  const hipError_t e = mmq::launch_quantize_q8_1(H, m.pairs(), m.F, q8, s);
  return e != hipSuccess ? e
                         : mmq::launch_moe_down(q8, plan, weights, w, residual, out, m, cus, s);
}

}  // namespace

extern "C" {

int mmq_moe_plan_bytes(int64_t M, int64_t E, int64_t k, size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  const int st = check_routing(M, E, k, true);
  if (st) return st;
  const mmq::MoeShape m{M, E, k, 0, 0};
  *bytes = (size_t)(4 * (mmq::kPlanHead + 4 * m.entries() + m.pairs()));
  return mmq::api_ok();
}

int mmq_moe_plan(int64_t M, int64_t E, int64_t k, const int32_t* ids, int32_t* plan,
                 void* stream) {
  int st = check_routing(M, E, k, true);
  if (!st) st = check_pointers({ids, plan});
  if (!st) st = mmq::api_current_device();
  if (st) return st;
  return hip_status("mmq_moe_plan",
                    mmq::launch_moe_plan(ids, M, E, k, plan, static_cast<hipStream_t>(stream)));
}

int mmq_moe_route(int64_t M, int64_t E, int64_t k, const float* logits, int32_t score,
                  int32_t renorm, int32_t* ids, float* weights, int32_t* plan, void* stream) {
  int st = check_routing(M, E, k, plan != nullptr);
  if (!st) st = check_route_options(score, renorm);
  if (!st) st = check_pointers({logits, ids, weights}, plan);
  if (!st) st = mmq::api_current_device();
  if (st) return st;
  return hip_status("mmq_moe_route",
                    mmq::launch_moe_route(logits, M, E, k, score, renorm, ids, weights, plan,
                                          static_cast<hipStream_t>(stream)));
}

int mmq_q4K_moe_gated(int64_t M, int64_t E, int64_t k, int64_t F, int64_t D, const float* x,
                      const int32_t* plan, const void* w_pairs, float* H, void* q8, int32_t act,
                      void* stream) {
  int st = check_gated(M, E, k, F, D, act);
  if (!st) st = check_pointers({x, plan, w_pairs, H, q8});
  if (!st) st = mmq::api_current_device();
  if (st) return st;
  return hip_status("mmq_q4K_moe_gated",
                    run_gated(mmq::MoeShape{M, E, k, D, F}, x, plan, w_pairs, H, q8, act,
                              static_cast<hipStream_t>(stream)));
}

int mmq_q4K_moe_down(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* H,
                     const int32_t* plan, const float* weights, const void* w_down,
                     const float* residual, float* out, void* q8, void* stream) {
  int st = check_down(M, E, k, D, F);
  const mmq::MoeShape m{M, E, k, D, F};
  int64_t cus = 0;
  if (!st) st = check_pointers({H, plan, weights, w_down, out, q8}, residual);
  if (!st) st = check_device(m, &cus);
  if (st) return st;
  return hip_status("mmq_q4K_moe_down",
                    run_down(m, H, plan, weights, w_down, residual, out, q8, cus,
                             static_cast<hipStream_t>(stream)));
}

int mmq_moe_workspace_bytes(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F,
                            size_t* bytes) {
  if (!bytes) return fail(MMQ_E_ARG, "bytes is NULL");
  int st = check_gated(M, E, k, F, D, MMQ_ACT_NONE);
  if (!st) st = check_down(M, E, k, D, F);
  if (st) return st;
  *bytes = (size_t)layout(M, E, k, D, F).total;
  return mmq::api_ok();
}

int mmq_q4K_moe(int64_t M, int64_t E, int64_t k, int64_t D, int64_t F, const float* x,
                const float* logits, int32_t score, int32_t renorm, const void* w_pairs,
                int32_t act, const void* w_down, const float* residual, float* out,
                void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gated(M, E, k, F, D, act);
  if (!st) st = check_down(M, E, k, D, F);
  if (!st) st = check_route_options(score, renorm);
  if (!st) st = check_pointers({x, logits, w_pairs, w_down, out, workspace}, residual);
  if (st) return st;
  const Workspace w = layout(M, E, k, D, F);
  if (workspace_bytes < (size_t)w.total)
    return fail(MMQ_E_ARG, "the layer needs %lld bytes of workspace, %llu given",
                (long long)w.total, (unsigned long long)workspace_bytes);
  const mmq::MoeShape m{M, E, k, D, F};
  int64_t cus = 0;
  if ((st = check_device(m, &cus))) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* ids = reinterpret_cast<int*>(ws + w.ids);
  float* weights = reinterpret_cast<float*>(ws + w.weights);
  int* plan = reinterpret_cast<int*>(ws + w.plan);
  float* H = reinterpret_cast<float*>(ws + w.H);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = mmq::launch_moe_route(logits, M, E, k, score, renorm, ids, weights, plan, s);
  if (e == hipSuccess) e = run_gated(m, x, plan, w_pairs, H, ws + w.q8, act, s);
  if (e == hipSuccess)
    e = run_down(m, H, plan, weights, w_down, residual, out, ws + w.q8, cus, s);
  return hip_status("mmq_q4K_moe", e);
}

}  // extern "C"
