// The router of a mixture-of-experts layer: per token the k experts of the greatest logits, their
// weights, and the plan that the experts' products read (moe_internal.h).
//
// One wavefront takes one token; lane l holds the logits of experts l, l + 64, .... A logit is
// compared as an unsigned key of the same order (0 for one that cannot be chosen: -inf, NaN, or
// past E), so a maximum over the wavefront is six v_max_u32 with lane moves, and k of them, each
// removing its winner, give the experts in order; among equal logits the lowest expert wins.
// Everything fits a few thousand cycles, so what bounds the call is its launch and one read of the
// logits; the plan is therefore made by the same launch for a few tokens: one workgroup then takes
// them all and sorts the pairs by expert from a bit matrix in LDS (expert x pair), whose bits are
// set with integer atomics (order-free) and counted. For more it is a launch of its own (launch_route).
#include "moe_internal.h"

namespace mmq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWords = (int)kMoeMaxPairs / 32;  // words of the bit matrix per expert
constexpr int kPlanPitch = kPlanWords + 1;          // odd: experts' words fall on distinct banks

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
// Maximum over the wavefront (row_shr 1, 2, 4, 8 within rows of 16 lanes, then the row
// broadcasts 15 and 31); lane 63 ends with it.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111>(v);
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);
  v = dpp_max<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111>(v);
  v = dpp_add<0x112>(v);
  v = dpp_add<0x114>(v);
  v = dpp_add<0x118>(v);
  v = dpp_add<0x142>(v);
  v = dpp_add<0x143>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// A float as an unsigned key of the same order; 0 for what cannot be chosen. -0 counts as 0.
__device__ __forceinline__ uint32_t key_of(float v, bool valid) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t key = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return valid && v == v && v > -INFINITY ? key : 0u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// e^(v - top), 1 at the top itself (an infinite top leaves the weight to its equals).
__device__ __forceinline__ float exp_below(float v, float top) {
  return v == top ? 1.0f : expf(v - top);
}

// The least float32 whose sigmoid is not 0 in float32: e^v rounds to 0 below 2^-150, v = -150 ln 2 =
// -103.972077. Below it normalised weights are 0: the sum of the scores is 0.
constexpr float kLeastSigmoid = -0x1.9fe368p+6f;

// One token. NV values per lane (E <= 64 NV). Lane s < k ends with slot s: its expert (-1: fewer
// than k could be chosen) and weight.
template <int NV>
__device__ void route_token(const float* __restrict__ logits, int E, int k, int score, bool renorm,
                            int lane, int& id, float& weight) {
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    key[i] = key_of(e < E ? logits[e] : 0.0f, e < E);
  }
  uint32_t kept[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) kept[i] = key[i];
  id = -1;
  uint32_t mine = 0;  // the key of this lane's slot
  uint32_t top = 0;
  for (int s = 0; s < k; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = key[i] > best ? key[i] : best;
    const uint32_t m = wave_max(best);
    if (m == 0) break;
    if (s == 0) top = m;
    // the lowest expert of that key: the first register that holds it, in its lowest lane
    int e = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint64_t has = __ballot(key[i] == m);
      if (e < 0 && has) e = 64 * i + (int)__builtin_ctzll(has);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 64 * i) key[i] = 0;
    if (lane == s) {
      id = e;
      mine = m;
    }
  }
  const float v = value_of(mine);
  if (score == 0) {
    const float t = value_of(top);
    weight = id >= 0 ? exp_below(v, t) : 0.0f;
    float all = weight;
    if (!renorm) {
      all = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) all += kept[i] ? exp_below(value_of(kept[i]), t) : 0.0f;
    }
    const float sum = wave_sum(all);
    weight = id >= 0 ? weight / sum : 0.0f;
  } else {
    // 1 / (1 + e^-v), for v < 0 as e^v / (1 + e^v): e^-v would overflow from 88.73 on. Normalised, the
    // factor e^-t of a negative greatest logit t cancels, so e^(v - t) / (1 + e^v) keeps the ratios
    // of scores that are themselves below float32's normal range.
    const float t = renorm ? fminf(value_of(top), 0.0f) : 0.0f;
    const float s = (v < 0.0f ? expf(v - t) : 1.0f) / (1.0f + expf(-fabsf(v)));
    weight = id >= 0 && t >= kLeastSigmoid ? s : 0.0f;
    if (renorm) {
      const float sum = wave_sum(weight);
      weight = sum > 0.0f ? weight / sum : 0.0f;
    }
  }
}

template <int NV>
__global__ __launch_bounds__(256) void route_kernel(const float* __restrict__ logits, int M, int E,
                                                    int k, int score, int renorm,
                                                    int* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int t = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  if (t >= M) return;
  int id;
  float w;
  route_token<NV>(logits + (size_t)t * E, E, k, score, renorm != 0, lane, id, w);
  if (lane < k) {
    ids[(size_t)t * k + lane] = id;
    weights[(size_t)t * k + lane] = w;
  }
}

struct PlanLds {
  uint32_t bits[kMoeMaxExperts * kPlanPitch];
  int ids[kMoeMaxPairs];
  int first[kMoeMaxExperts];
  uint32_t wave_total[kPlanThreads / 64];
};

// The plan of sh.ids[0..P) (written, with a barrier behind it), by a workgroup of kPlanThreads.
__device__ void make_plan(PlanLds& sh, int P, int E, int* __restrict__ plan) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int words = (P + 31) >> 5;
  const int entries = E < P ? E : P;
  for (int i = tid; i < E * kPlanPitch; i += kPlanThreads) sh.bits[i] = 0;
  __syncthreads();
  const int id = tid < P ? sh.ids[tid] : -1;
  const bool valid = id >= 0 && id < E;
  if (valid) atomicOr(&sh.bits[id * kPlanPitch + (tid >> 5)], 1u << (tid & 31));
  __syncthreads();
  // pairs of expert tid, and the running sums of (pairs, used) packed as pairs | used << 16
  uint32_t own = 0;
  if (tid < E)
    for (int w = 0; w < words; ++w) own += (uint32_t)__popc(sh.bits[tid * kPlanPitch + w]);
  own |= own ? 1u << 16 : 0u;
  uint32_t incl = own;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) sh.wave_total[wave] = incl;
  __syncthreads();
  uint32_t before = 0, total = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const uint32_t v = sh.wave_total[w];
    if (w < wave) before += v;
    total += v;
  }
  const uint32_t excl = before + incl - own;
  const int n = (int)(own & 0xFFFFu), first = (int)(excl & 0xFFFFu), rank = (int)(excl >> 16);
  const int pairs = (int)(total & 0xFFFFu), used = (int)(total >> 16);
  int4* entry = reinterpret_cast<int4*>(plan + kPlanHead);
  if (tid < E) sh.first[tid] = first;
  if (n > 0) entry[rank] = make_int4(tid, first, n, 0);
  if (tid >= used && tid < entries) entry[tid] = make_int4(-1, 0, 0, 0);
  if (tid == 0) *reinterpret_cast<int4*>(plan) = make_int4(used, pairs, 0, 0);
  __syncthreads();
  int* order = plan + kPlanHead + 4 * entries;
  if (valid) {  // its place: how many of its expert's pairs come before it
    const uint32_t* b = sh.bits + id * kPlanPitch;
    int at = sh.first[id] + __popc(b[tid >> 5] & ((1u << (tid & 31)) - 1u));
    for (int w = 0; w < (tid >> 5); ++w) at += __popc(b[w]);
    order[at] = tid;
  }
  if (tid >= pairs && tid < P) order[tid] = -1;
}

template <int NV>
__global__ __launch_bounds__(kPlanThreads) void route_plan_kernel(
    const float* __restrict__ logits, int M, int E, int k, int score, int renorm,
    int* __restrict__ ids, float* __restrict__ weights, int* __restrict__ plan) {
  __shared__ PlanLds sh;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = wave; t < M; t += kPlanThreads / 64) {
    int id;
    float w;
    route_token<NV>(logits + (size_t)t * E, E, k, score, renorm != 0, lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      weights[t * k + lane] = w;
      sh.ids[t * k + lane] = id;
    }
  }
  __syncthreads();
  make_plan(sh, M * k, E, plan);
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int* __restrict__ ids, int P,
                                                            int E, int* __restrict__ plan) {
  __shared__ PlanLds sh;
  if ((int)threadIdx.x < P) sh.ids[threadIdx.x] = ids[threadIdx.x];
  __syncthreads();
  make_plan(sh, P, E, plan);
}

template <int NV>
hipError_t launch_route(const float* logits, int64_t M, int64_t E, int64_t k, int score, int renorm,
                        int* ids, float* weights, int* plan, hipStream_t s) {
  // One launch for both while the plan's one workgroup has few tokens per wavefront to route: graph
  // replays, one launch against two, 4.9 / 6.5 us for 16 tokens of 64 experts, 6.7 / 7.5 for 16 of
  // 256, but 10.0 / 7.6 for 32 of 256, 10.2 / 6.9 for 64 of 64 and 16.6 / 7.8 for 64 of 256.
  if (plan && M * (NV + 1) > 96) {
    const hipError_t e =
        launch_route<NV>(logits, M, E, k, score, renorm, ids, weights, nullptr, s);
    return e != hipSuccess ? e : launch_moe_plan(ids, M, E, k, plan, s);
  }
  if (plan)
    hipLaunchKernelGGL(route_plan_kernel<NV>, dim3(1), dim3(kPlanThreads), 0, s, logits, (int)M,
                       (int)E, (int)k, score, renorm, ids, weights, plan);
  else
    hipLaunchKernelGGL(route_kernel<NV>, dim3((unsigned)((M + 3) / 4)), dim3(256), 0, s, logits,
                       (int)M, (int)E, (int)k, score, renorm, ids, weights);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const float* logits, int64_t M, int64_t E, int64_t k, int score,
                            int renorm, int* ids, float* weights, int* plan, hipStream_t s) {
  if (E <= 64) return launch_route<1>(logits, M, E, k, score, renorm, ids, weights, plan, s);
  if (E <= 128) return launch_route<2>(logits, M, E, k, score, renorm, ids, weights, plan, s);
  if (E <= 256) return launch_route<4>(logits, M, E, k, score, renorm, ids, weights, plan, s);
  return launch_route<8>(logits, M, E, k, score, renorm, ids, weights, plan, s);
}

hipError_t launch_moe_plan(const int* ids, int64_t M, int64_t E, int64_t k, int* plan,
                           hipStream_t s) {
  hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, ids, (int)(M * k), (int)E,
                     plan);
  return hipGetLastError();
}

}  // namespace mmq
