// Matrix-vector products with 4-bit weights and one scale (and zero) per group of values, for 1 to 16
// tokens:
//
//   y[i][j] = act( sum_g s_jg ( sum_{k in g} x_ik v_jk - z_jg sum_{k in g} x_ik ) + bias_j ) + res_ij
//
// The nibbles v are exact in f16 and bf16, and so is every product x v in float32, so the inner sums
// run on v_mfma_f32_16x16x32_{f16,bf16} with float32 accumulators: 16 weight rows (src0) by 16
// columns (src1). A float16 or bfloat16 token is one column. A float32 token is three: its values'
// three bf16 pieces, which sum to them exactly (bf16_trunc3), so nothing is rounded before the
// float32 sums, whatever the type. sum x is the same instruction with a row of ones, and lands where
// the fold needs it. The zero stays out of the operand (a zero need not be a whole number) and costs
// two FMAs per group and result.
//
// Bound by the bytes of the weights: a workgroup has 16 rows, its wavefronts take the records of 128
// values in turn (so that together they stream contiguous memory), load kBatch of them ahead, and
// add their sums through LDS in the order of the wavefronts. The matrix instructions are idle most
// of the time with few tokens; what counts beside the loads is unpacking: 9 vector instructions per
// 8 values to f16 (or the exponent of 1024 over the nibble, subtract 1024), 15 to bf16 (convert
// bytes to float32, keep the high halves).
#include <type_traits>

#include "epilogue.h"
#include "mmq_device.h"
#include "q4g_internal.h"

namespace mmq {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kBatch = 2;                 // records a wavefront loads ahead
constexpr int kPitch = kG4Values * 2 + 16;  // LDS bytes per column of pieces: 16-byte reads spread

// Columns of 16 that M tokens make.
constexpr int columns(int x_type, int64_t M) { return (int)(x_type == kTypeF32 ? 3 * M : M); }
constexpr int column_tiles(int x_type, int64_t M) { return (columns(x_type, M) + 15) / 16; }

// The eight values of a dword as the matrix operand, four registers of two.
template <bool BF>
__device__ __forceinline__ v4u unpack(uint32_t w) {
  v4u o;
  if constexpr (BF) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // nibbles j and j + 4
      const uint32_t b = j & 1 ? hi : lo;
      const int at = 8 * (j >> 1);
      const float a = (float)((b >> at) & 0xFFu), c = (float)((b >> (at + 16)) & 0xFFu);
      o[j] = pack_hi16(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, c));
    }
  } else {
    // 0x6400 | v is 1024 + v and 0x5400 | v << 4 is 64 + v, exactly
    const uint32_t w8 = w >> 8;
    const v2h big = {(_Float16)1024.0f, (_Float16)1024.0f}, mid = {(_Float16)64.0f, (_Float16)64.0f};
    const uint32_t p[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x54005400u,
                           (w8 & 0x000F000Fu) | 0x64006400u, (w8 & 0x00F000F0u) | 0x54005400u};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, p[j]) - (j & 1 ? mid : big));
  }
  return o;
}

template <bool BF>
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <bool SBF>
__device__ __forceinline__ float scale_of(uint2 u, int r) {
  const uint32_t w = r & 2 ? u.y : u.x;
  if constexpr (SBF)
    return __builtin_bit_cast(float, r & 1 ? w & 0xFFFF0000u : w << 16);
  else
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(r & 1 ? w >> 16 : w));
}

__device__ __forceinline__ float load_as_float(const void* p, size_t i, int type) {
  if (type == kTypeF32) return static_cast<const float*>(p)[i];
  if (type == kTypeF16) return (float)static_cast<const _Float16*>(p)[i];
  return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ void store_float(void* p, size_t i, int type, float v) {
  if (type == kTypeF32) static_cast<float*>(p)[i] = v;
  else if (type == kTypeF16) static_cast<_Float16*>(p)[i] = (_Float16)v;  // nearest, ties to even
  else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

// XT: the tokens' type. CT: column tiles. FOLDS: folds of a record, 1 where its 128 values lie in one
// group, else 4, one per 32 values. SBF: bf16 scales.
template <int XT, int CT, int FOLDS, bool ZEROS, bool SBF, int NW>
__global__ __launch_bounds__(64 * NW) void q4g_kernel(const void* __restrict__ x,
                                                      const uint8_t* __restrict__ rep, void* y,
                                                      int y_type, int M, int N, int K, int group,
                                                      size_t scales_at, size_t zeros_at,
                                                      Q4GEpilogue epi) {
  constexpr bool F32 = XT == kTypeF32;
  constexpr bool BF = XT != kTypeF16;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane >> 4, l16 = lane & 15;
  const int tile = blockIdx.x;
  const int nrec = (K + kG4Values - 1) / kG4Values;
  const int ngroups = (K + group - 1) / group;
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(rep + (size_t)tile * nrec * kG4RecBytes, (uint32_t)nrec * kG4RecBytes);
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(rep + scales_at + (size_t)tile * ngroups * 32, (uint32_t)ngroups * 32);
  const __amdgpu_buffer_rsrc_t rz =
      make_rsrc(rep + zeros_at + (size_t)tile * ngroups * 32, ZEROS ? (uint32_t)ngroups * 32 : 0u);
  constexpr uint32_t XB = F32 ? 4 : 2;
  const uint32_t x_bytes = (uint32_t)M * (uint32_t)K * XB;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x, x_bytes);

  struct Rec {
    v4i w;
    uint2 s[FOLDS], z[ZEROS ? FOLDS : 1];
    v4u x[F32 ? 1 : 4];                      // 16-bit tokens: the operands of the four steps
    float2 f[F32 ? (16 * CT + 2) / 3 : 1];   // float32: two values of each token
  };
  constexpr int MT = F32 ? (16 * CT) / 3 : 0;  // float32 tokens that CT column tiles hold
  auto load = [&](Rec& r, int rec) {
    // past the last record every offset is past its buffer, and reads 0
    const uint32_t o = (uint32_t)min(rec, nrec);
    r.w = buf_load16_aux<kReadOnce>(rw, o * kG4RecBytes + lane * 16);
#pragma unroll
    for (int i = 0; i < FOLDS; ++i) {
      const int k0 = (int)o * kG4Values + 32 * i;
      const uint32_t at = k0 < K ? (uint32_t)(k0 / group) * 32u + c * 8 : 0x7FFFFFF0u;
      r.s[i] = buf_load8_aux<0>(rs, at);
      if constexpr (ZEROS) r.z[i] = buf_load8_aux<0>(rz, at);
    }
    if constexpr (F32) {
      const uint32_t k = o * kG4Values + 2 * lane;
#pragma unroll
      for (int t = 0; t < MT; ++t)
        r.f[t] = t < M && (int)k < K
                     ? buf_load_f32x2(rx, ((uint32_t)t * (uint32_t)K + k) * 4u)
                     : make_float2(0.f, 0.f);
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t k = o * kG4Values + 32 * m;
        const uint32_t at = l16 < M && (int)k < K
                                ? ((uint32_t)l16 * (uint32_t)K + k + 8 * c) * 2u
                                : x_bytes;
        r.x[m] = __builtin_bit_cast(v4u, buf_load16(rx, at));
      }
    }
  };

  v4f out[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) out[ct] = v4f{0.f, 0.f, 0.f, 0.f};
  const v4u ones = BF ? v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}
                      : v4u{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
  uint8_t* cols = smem + wave * (16 * CT * kPitch);  // this wavefront's pieces, [column][128]

  auto compute = [&](const Rec& r) {
    if constexpr (F32) {
      // the pieces of two values of each token; only this wavefront uses the region, and its LDS
      // operations are in order, so the reads of the record before are done
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (t < M) {
          uint32_t a[3], b[3];
          bf16_trunc3(r.f[t].x, a[0], a[1], a[2]);
          bf16_trunc3(r.f[t].y, b[0], b[1], b[2]);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint32_t*>(cols + (3 * t + i) * kPitch + lane * 4) =
                pack_hi16(a[i], b[i]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    v4f acc[CT], xs[CT];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const v4u wv = unpack<BF>((uint32_t)r.w[m]);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        v4u xv;
        if constexpr (F32)
          xv = *reinterpret_cast<const v4u*>(cols + (16 * ct + l16) * kPitch + m * 64 + c * 16);
        else
          xv = r.x[m];
        const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
        const bool first = m == 0 || FOLDS == 4;
        acc[ct] = mfma<BF>(wv, xv, first ? zero : acc[ct]);
        xs[ct] = mfma<BF>(ones, xv, first ? zero : xs[ct]);
      }
      if (FOLDS == 4 || m == 3) {
        const int i = FOLDS == 4 ? m : 0;
#pragma unroll
        for (int rr = 0; rr < 4; ++rr) {
          const float sc = scale_of<SBF>(r.s[i], rr);
          const float z = ZEROS ? scale_of<SBF>(r.z[ZEROS ? i : 0], rr) : 8.0f;
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            out[ct][rr] =
                __builtin_fmaf(sc, __builtin_fmaf(-z, xs[ct][rr], acc[ct][rr]), out[ct][rr]);
        }
      }
    }
    if constexpr (F32) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  };

  Rec cur[kBatch], nxt[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) load(cur[u], wave + u * NW);
  for (int rec = wave; rec < nrec; rec += kBatch * NW) {
    const bool more = rec + kBatch * NW < nrec;
    if (more) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) load(nxt[u], rec + (kBatch + u) * NW);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) compute(cur[u]);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) cur[u] = nxt[u];
  }

  // The wavefronts' sums, [wave][column][16 rows], added in the order of the wavefronts; a float32
  // token's three columns after that, the largest last.
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
    *reinterpret_cast<float4*>(red + ((wave * CT + ct) * 16 + l16) * 16 + 4 * c) =
        make_float4(out[ct][0], out[ct][1], out[ct][2], out[ct][3]);
  __syncthreads();
  for (int i = tid; i < 16 * M; i += 64 * NW) {
    const int t = i >> 4, row = i & 15;
    const int j = tile * kG4Rows + row;
    if (j >= N) continue;
    auto total = [&](int col) {
      float v = red[col * 16 + row];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += red[(w * CT * 16 + col) * 16 + row];
      return v;
    };
    float v;
    if constexpr (F32) v = (total(3 * t + 2) + total(3 * t + 1)) + total(3 * t);
    else v = total(t);
    if (epi.bias) v += epi.bias[j];
    v = activate(v, epi.act);
    const size_t at = (size_t)t * N + j;
    if (epi.residual) v += load_as_float(epi.residual, at, y_type);
    store_float(y, at, y_type, v);
  }
}

constexpr int64_t lds_bytes(int x_type, int ct, int nw) {
  const int64_t red = (int64_t)nw * ct * 16 * 16 * 4;
  const int64_t cols = x_type == kTypeF32 ? (int64_t)nw * 16 * ct * kPitch : 0;
  return red > cols ? red : cols;
}

// Wavefronts of a workgroup.
int wavefronts(const Q4GShape&, int64_t) { return 8; }

struct Call {
  const void* x;
  const uint8_t* rep;
  void* y;
  int y_type;
  int64_t M;
  Q4GShape g;
  Q4GEpilogue epi;
};

template <int XT, int CT, int FOLDS, bool ZEROS, bool SBF, int NW>
hipError_t launch_t(const Call& c, hipStream_t s) {
  auto kern = q4g_kernel<XT, CT, FOLDS, ZEROS, SBF, NW>;
  constexpr int64_t lds = lds_bytes(XT, CT, NW);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const int group = (int)(c.g.group < c.g.K ? c.g.group : c.g.K);
  hipLaunchKernelGGL(kern, dim3((unsigned)c.g.tiles()), dim3(64 * NW), (size_t)lds, s, c.x, c.rep,
                     c.y, c.y_type, (int)c.M, (int)c.g.N, (int)c.g.K, group,
                     (size_t)c.g.scales_at(), (size_t)c.g.zeros_at(), c.epi);
  return hipGetLastError();
}

template <int XT, int CT, int NW>
hipError_t launch_type(const Call& c, int scale_type, hipStream_t s) {
  const bool one = c.g.group % kG4Values == 0 || c.g.group >= c.g.K;
  const bool sbf = scale_type == kTypeBF16;
  auto pick = [&](auto z, auto b) {
    constexpr bool Z = decltype(z)::value, B = decltype(b)::value;
    return one ? launch_t<XT, CT, 1, Z, B, NW>(c, s) : launch_t<XT, CT, 4, Z, B, NW>(c, s);
  };
  constexpr std::integral_constant<bool, true> yes{};
  constexpr std::integral_constant<bool, false> no{};
  return c.g.zeros ? (sbf ? pick(yes, yes) : pick(yes, no)) : (sbf ? pick(no, yes) : pick(no, no));
}

template <int NW>
hipError_t launch_nw(const Call& c, int x_type, int scale_type, hipStream_t s) {
  if (x_type == kTypeF16) return launch_type<kTypeF16, 1, NW>(c, scale_type, s);
  if (x_type == kTypeBF16) return launch_type<kTypeBF16, 1, NW>(c, scale_type, s);
  switch (column_tiles(kTypeF32, c.M)) {
    case 1: return launch_type<kTypeF32, 1, NW>(c, scale_type, s);
    case 2: return launch_type<kTypeF32, 2, NW>(c, scale_type, s);
    default: return launch_type<kTypeF32, 3, NW>(c, scale_type, s);
  }
}

// One work-item per dword of the values, one per scale and per zero.
__global__ __launch_bounds__(256) void repack_values_kernel(const uint8_t* __restrict__ w,
                                                            uint32_t* __restrict__ rep, int64_t N,
                                                            int64_t K, int64_t nrec, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t at = i >> 8;  // (tile, record)
  const int64_t tile = at / nrec, rec = at - tile * nrec;
  const int q = (int)(i & 255), m = q & 3, row = (q >> 2) & 15, c = q >> 6;
  const int64_t j = tile * kG4Rows + row, k = rec * kG4Values + 32 * m + 8 * c;
  uint32_t o = 0;
  if (j < N && k < K) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(w + (j * K + k) / 2);
    // nibble e of v (value e) goes to nibble e / 2 + 4 (e % 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) o |= ((v >> (4 * e)) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
  }
  rep[i] = o;
}
__global__ __launch_bounds__(256) void repack_scales_kernel(const uint16_t* __restrict__ s,
                                                            uint16_t* __restrict__ rep, int64_t N,
                                                            int64_t ngroups, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t at = i >> 4;  // (tile, group)
  const int64_t tile = at / ngroups, g = at - tile * ngroups;
  const int64_t j = tile * kG4Rows + (i & 15);
  rep[i] = j < N ? s[j * ngroups + g] : (uint16_t)0;
}

}  // namespace

int64_t q4g_lds_bytes(int x_type, int64_t M, const Q4GShape& g, int64_t compute_units) {
  return lds_bytes(x_type, column_tiles(x_type, M), wavefronts(g, compute_units));
}

hipError_t launch_q4g(const void* x, int x_type, const void* rep, int scale_type, void* y,
                      int y_type, int64_t M, const Q4GShape& g, const Q4GEpilogue& epi,
                      int64_t compute_units, hipStream_t s) {
  const Call c{x, static_cast<const uint8_t*>(rep), y, y_type, M, g, epi};
  (void)compute_units;
  return launch_nw<8>(c, x_type, scale_type, s);
}

hipError_t launch_repack_q4g(const void* w, const void* scales, const void* zeros,
                             const Q4GShape& g, void* rep, hipStream_t s) {
  uint8_t* base = static_cast<uint8_t*>(rep);
  const int64_t n = g.scales_at() / 4, ns = g.tiles() * g.groups() * 16;
  hipLaunchKernelGGL(repack_values_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     static_cast<const uint8_t*>(w), reinterpret_cast<uint32_t*>(base), g.N, g.K,
                     g.records(), n);
  hipError_t e = hipGetLastError();
  for (int i = 0; e == hipSuccess && i < (g.zeros ? 2 : 1); ++i) {
    hipLaunchKernelGGL(repack_scales_kernel, dim3((unsigned)((ns + 255) / 256)), dim3(256), 0, s,
                       static_cast<const uint16_t*>(i ? zeros : scales),
                       reinterpret_cast<uint16_t*>(base + (i ? g.zeros_at() : g.scales_at())), g.N,
                       g.groups(), ns);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace mmq
