// The mixture-of-experts kernels' shared declarations (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

// Limits of the plan and of the kernels that read it.
constexpr int64_t kMoeMaxTokens = 64;
constexpr int64_t kMoeMaxPairs = 512;
constexpr int64_t kMoeMaxExperts = 512;

// The plan, int32: [used experts, pairs, 0, 0], then min(E, M*k) entries [expert, first, pairs, 0]
// (the used experts in increasing order, then entries of no pairs), then the M*k pairs sorted by
// expert (those of no expert, -1, last).
constexpr int kPlanHead = 4;

struct MoeShape {
  int64_t M, E, k;  // tokens, experts, slots per token
  int64_t D, F;     // model width and the experts' inner width
  int64_t pairs() const { return M * k; }
  int64_t entries() const { return E < M * k ? E : M * k; }
};

struct PlanEntry {
  int expert, first, n;
};
// Entry u, of no pairs unless the plan's numbers are inside its own sizes.
__device__ __forceinline__ PlanEntry plan_entry(const int* plan, int u, int E, int P) {
  const int4 v = *reinterpret_cast<const int4*>(plan + kPlanHead + 4 * u);
  PlanEntry e{v.x, v.y, v.z};
  if (e.expert < 0 || e.expert >= E || e.first < 0 || e.n < 0 || e.first > P || e.n > P - e.first)
    e = PlanEntry{0, 0, 0};
  return e;
}

hipError_t launch_moe_route(const float* logits, int64_t M, int64_t E, int64_t k, int score,
                            int renorm, int* ids, float* weights, int* plan, hipStream_t s);
hipError_t launch_moe_plan(const int* ids, int64_t M, int64_t E, int64_t k, int* plan,
                           hipStream_t s);
// H[M*k][F] from E matrices of pair records (F, D) and `tokens`: x itself, float32, where the
// kernel quantizes it (moe_fused), else the q8 buffer of x (M x D).
hipError_t launch_moe_gated(const void* tokens, const int* plan, const void* w, float* H,
                            const MoeShape& m, int act, hipStream_t s);
// out[M][D] from E matrices of repacked records (D, F) and `tokens`: H or its q8 buffer (M*k x F).
hipError_t launch_moe_down(const void* tokens, const int* plan, const float* weights,
                           const void* w, const float* residual, float* out, const MoeShape& m,
                           int64_t compute_units, hipStream_t s);
int64_t moe_down_lds_bytes(const MoeShape& m, int64_t compute_units);
// Whether the products quantize their own activations: with one token each expert has one column.
inline bool moe_fused(int64_t M) { return M == 1; }

}  // namespace mmq
