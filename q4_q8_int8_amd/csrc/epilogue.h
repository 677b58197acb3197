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
// All of it is float32, as the products are. It runs at the end of a kernel, on sums that are in
// registers: vector instructions, and with a residual one more read of the output's size, asked for
// ahead of the sums. Six of one product behind one another in a graph, on one set of weights: 2048 x
// 4096 x 4096 takes 91.7 us plain, 91.9 with a residual (a torch addition behind the product: 105.0),
// 97.1 with bias, gelu and a residual; 2048 x 11008 x 4096 gated with silu 485 us, against 489 for the
// product of the same 22016 rows alone, which writes twice the bytes. (Between other kernels, as in a
// trace of whole calls, the gated one takes 495 to 523.)
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

// v / (1 + e^-u), without overflow: e = e^-|u| is in (0, 1]. The exponential and the reciprocal are
// the hardware's (1 unit in the last place each; results below 2^-126 are 0), so the quotient is
// good to a few units; the rounding of u log2(e) is one of u, which reaches the result as
// |v u s (1 - s)| half units, s = 1 / (1 + e^-u).
__device__ __forceinline__ float times_sigmoid(float v, float u) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(u) * -1.44269504f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return v * (u >= 0.0f ? r : e * r);
}

// gelu(v) = v Phi(v), Phi the normal distribution, from its upper tail Q(t) = Phi(-t), t = |v|:
// v (1 - Q) for v >= 0, v Q below, so that neither side cancels. Q(t) = e^(-t^2/2) R(t) with the
// smooth R(t) = e^(t^2/2) Phi(-t), fitted (least squares iterated to an equal ripple) by s p(s), s =
// 1 / (1 + 3/8 t), p of degree 8, to 2.5e-7 of R over 0 <= t < 660: at most 4e-8 of max(1, |v|) in
// gelu. (The library's erfc, with its branches, is about 80 instructions, this about 20: 2048 x 22016
// outputs took 77 us more with it.)
__device__ __forceinline__ float gelu_erf(float v) {
  const float t = __builtin_fabsf(v);
  const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(t, 0.375f, 1.0f));
  float p = -0.032911047f;
  p = __builtin_fmaf(p, s, 0.13687992f);
  p = __builtin_fmaf(p, s, -0.18652119f);
  p = __builtin_fmaf(p, s, 0.050632391f);
  p = __builtin_fmaf(p, s, 0.015627913f);
  p = __builtin_fmaf(p, s, 0.088638239f);
  p = __builtin_fmaf(p, s, 0.12844568f);
  p = __builtin_fmaf(p, s, 0.14960459f);
  p = __builtin_fmaf(p, s, 0.14960338f);
  const float q = __builtin_amdgcn_exp2f(t * t * -0.72134752f) * (p * s);
  return v * (v >= 0.0f ? 1.0f - q : q);
}

// act(v); NaN passes all of them.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActSilu: return times_sigmoid(v, v);
    case kActGelu: return gelu_erf(v);
    case kActGeluTanh:  // the tanh form is v / (1 + e^-2u), u = sqrt(2/pi) (v + 0.044715 v^3)
      return times_sigmoid(v, v * __builtin_fmaf(v * v, 0.071354816f, 1.5957691216f));
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

// Four consecutive elements, at a 16-byte aligned place: what they need from memory, which a kernel
// may ask for ahead of their sums, and the result.
template <int EPI>
__device__ __forceinline__ float4 epi_bias(const EpiParam<EPI>& e, int j) {
  float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if constexpr (EPI == kEpiAct)
    if (e.bias) b = *reinterpret_cast<const float4*>(e.bias + j);
  return b;
}
template <int EPI>
__device__ __forceinline__ float4 epi_residual(const EpiParam<EPI>& e, size_t at) {
  float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if constexpr (EPI == kEpiAct)
    if (e.residual) r = *reinterpret_cast<const float4*>(e.residual + at);
  return r;
}
template <int EPI>
__device__ __forceinline__ float4 epi_four(const EpiParam<EPI>& e, float4 v, float4 b, float4 r) {
  if constexpr (EPI == kEpiAct) {
    if (e.bias) {
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    if (e.act != kActNone) {
      v.x = activate(v.x, e.act); v.y = activate(v.y, e.act);
      v.z = activate(v.z, e.act); v.w = activate(v.w, e.act);
    }
    if (e.residual) {
      v.x += r.x; v.y += r.y; v.z += r.z; v.w += r.w;
    }
  }
  return v;
}

}  // namespace mmq
