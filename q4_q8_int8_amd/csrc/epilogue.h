// The epilogue of the products (not part of the ABI): what a kernel does with an output element
// after its last partial sum has been added, and the host's description of it.
//
//   kEpiNone    C = P
//   kEpiAct     C = act(P + bias) + residual          (bias and residual may be absent)
//   kEpiGated   H = act(G) * U, from weights whose rows alternate, 8 of the gate and 8 of the up
//               matrix (the pair records of repack_q4_K_pair): packed row 16 b + r, r < 8, is row
//               8 b + r of the gate, and 16 b + 8 + r the same row of the up matrix. In every
//               kernel's result layout the two then sit in one lane's registers, or in one
//               workgroup's 16 rows, so neither product goes through memory.
//
// All of it is float32, as the products are. The epilogue costs one activation per output, next to
// K / 32 rescales per output in the product itself, so it is evaluated with the accurate library
// functions (expf, erfcf) rather than the fast intrinsics.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

constexpr int kEpiNone = 0;
constexpr int kEpiAct = 1;
constexpr int kEpiGated = 2;

// enum mmq_act, restated for the kernels
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

// The host's description of an epilogue, handed to the launchers.
struct Epilogue {
  int kind = kEpiNone;
  int act = kActNone;
  const float* bias = nullptr;
  const float* residual = nullptr;
  int64_t F = 0;  // kEpiGated: columns of H (the product's N is then the packed row count)
};

// What a kernel takes of it.
template <int EPI>
struct EpiParam {};
template <>
struct EpiParam<kEpiAct> {
  const float* bias;
  const float* residual;
  int act;
};
template <>
struct EpiParam<kEpiGated> {
  int act;
  int F;
};

template <int EPI>
inline EpiParam<EPI> epi_param(const Epilogue& e) {
  if constexpr (EPI == kEpiAct) return {e.bias, e.residual, e.act};
  else if constexpr (EPI == kEpiGated) return {e.act, (int)e.F};
  else return {};
}

// Packed rows of a pair of matrices with F rows each: whole 32-row tiles of 16 + 16.
__host__ __device__ constexpr int64_t pair_rows(int64_t F) { return (F + 15) / 16 * 32; }

// act(v). silu(v) = v / (1 + e^-v) and gelu_tanh(v) = v / (1 + e^-2u), u = sqrt(2/pi)(v +
// 0.044715 v^3), the tanh form of the same function without its cancellation at negative v. Where
// e^-v overflows the quotient is -0, the limit; -inf gives NaN as -inf * 0 does. gelu(v) = v/2
// erfc(-v/sqrt 2): erfc keeps its relative precision where 1 + erf would cancel.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case kActRelu: return v < 0.0f ? 0.0f : v;  // NaN passes
    case kActSilu: return v / (1.0f + expf(-v));
    case kActGelu: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case kActGeluTanh: {
      const float u2 = v * __builtin_fmaf(v * v, 0.071354816f, 1.5957691216f);
      return v / (1.0f + expf(-u2));
    }
    default: return v;
  }
}

// C[i][j] of an M x N output from its finished sum. `at` is i * N + j. A residual may be C itself:
// the element is read here, by the work-item that then stores it.
template <int EPI>
__device__ __forceinline__ float epi_one(const EpiParam<EPI>& e, float v, size_t at, int j) {
  if constexpr (EPI == kEpiAct) {
    if (e.bias) v += e.bias[j];
    v = activate(v, e.act);
    if (e.residual) v += e.residual[at];
  }
  return v;
}

// Four consecutive elements, at a 16-byte aligned place.
template <int EPI>
__device__ __forceinline__ float4 epi_four(const EpiParam<EPI>& e, float4 v, size_t at, int j) {
  if constexpr (EPI == kEpiAct) {
    if (e.bias) {
      const float4 b = *reinterpret_cast<const float4*>(e.bias + j);
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    if (e.act != kActNone) {
      v.x = activate(v.x, e.act); v.y = activate(v.y, e.act);
      v.z = activate(v.z, e.act); v.w = activate(v.w, e.act);
    }
    if (e.residual) {
      const float4 r = *reinterpret_cast<const float4*>(e.residual + at);
      v.x += r.x; v.y += r.y; v.z += r.z; v.w += r.w;
    }
  }
  return v;
}

}  // namespace mmq
