// Matrix-vector products with 4-bit weights and one scale (and zero) per group of values, for 1 to 16
// tokens:
//
//   y[i][j] = act( sum_g s_jg ( sum_{k in g} x_ik v_jk - z_jg sum_{k in g} x_ik ) + bias_j ) + res_ij
//
// The inner sums run on v_mfma_f32_16x16x32_{f16,bf16} with float32 accumulators: src0 has 16 columns
// of activations, src1 16 weight rows, so a lane's four results are of one weight row and share its
// scale. Every product is exact in float32: a nibble is exact in f16; for bf16 the operand is 16 + v
// (the bits of 16 with v in the upper mantissa bits, one AND-OR behind a shift), and the 16 goes out
// with the zero, - (16 + z) sum x. That operand and the ones below come with a factor of 2^-12, which
// an output's sum is freed of at its end: 128 x 31 x 2^-12 is below 1, so that no sum of a record
// overflows where its terms, of either sign and larger than those of v - z, would, whatever finite
// values a token has (the bits are those without the factor, but for sums below 2^-114, which get an
// error of 2^-137 for each of their terms). A float16 or bfloat16 token is one column, token t being column
// 4 (t % 4) + t / 4, so that up to four tokens need one result register. A float32 token is three
// columns, its values' three bf16 pieces, which sum to them exactly (bf16_trunc3): token t has columns
// 4 (t % 4) .. + 2 of column tile t / 4, so that its three sums meet in one lane. sum x is the same
// instruction with ones for weights; the matrix unit is idle most of the time.
//
// Bound by the bytes of the weights. A workgroup, one to a compute unit, works through tiles of 16 rows; its
// wavefronts take the records of 128 values in turn (together they stream contiguous memory), each with
// kAhead records in flight, across the tiles too. Their sums of several tiles are added together, through
// LDS, in the order of the wavefronts: a barrier for every tile costs as much as a tile's loads. A
// wavefront brings the values of x for its own records into LDS with its first tile, in the form of the
// operands: read from memory for every tile they take more of the vector memory unit than the weights do,
// and their latency is not covered (16 tokens, 11008 x 4096: 16.3 us in a graph, 11.5 from LDS). Beside the
// loads, unpacking counts: 9 vector instructions per 8 values for f16 and 8 for bf16. Where x of a wavefront's
// records does not fit the LDS it is brought in for one record at a time, anew for every tile, behind a wait that
// the weights in flight end with too: 16 x 8192 x 8192 bf16 15.7 us (36 MB), 16 x 28672 x 8192 46.9 (125 MB); for
// float32 tokens from 7 on at K = 4096, 16 x 11008 x 4096 24.5 (24 MB). With 9 float32 tokens or more and four
// scales a record the kernel spills 57 registers with x in LDS, 2 without (27.6 us).
//
// Graph replays over weights beyond the caches, a launch being 3.6 us of each: 1 x 4096 x 4096 f16 5.1 us (9 MB),
// 1 x 4096 x 11008 f32 with groups of 32 and zeros 11.1 (28 MB), 16 x 11008 x 4096 bf16 11.4 (24 MB),
// 1 x 22016 x 4096 bf16 13.1 (48 MB): 3.1 to 6 TB/s beyond the launch, VALU 33 to 54 % busy.
#include <algorithm>

#include "epilogue.h"
#include "mmq_device.h"
#include "q4g_internal.h"

namespace mmq {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kAhead = 4;              // records of a wavefront in flight, per tile
constexpr int kRowBytes = kG4Values * 2;  // LDS bytes of a row of a record's operands
// Wavefronts of a workgroup at most: the sums of many float32 tokens take registers.
constexpr int max_waves(int x_type, int q) { return x_type == kTypeF32 && q > 1 ? 8 : 16; }
// The rows of x in LDS: of each token one, or three of pieces.
__host__ __device__ constexpr int x_rows(int x_type, int64_t M) {
  return (int)(x_type == kTypeF32 ? 3 * M : M);
}
// Where the 16 bytes `part` (0..15) of a row are: moved about by the row, so that the same part of
// neighbouring rows is in different banks.
__device__ __forceinline__ int x_place(int row, int part) {
  return row * kRowBytes + ((part ^ (row & 15)) * 16);
}

// 16 bytes at a lane's offset from a wavefront's.
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, lane_at, at, 0));
}

// Constants that stay in vector registers, where an AND-OR can take them beside a mask in scalar ones (the
// compiler would otherwise spend two instructions with literals).
__device__ __forceinline__ uint32_t keep(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The eight values of a dword as the matrix operand, four registers of two: v for f16, 2^-12 (16 + v) for
// bf16, and the 1 (2^-12) that sums x.
template <bool BF>
struct Unpack;
template <>
struct Unpack<true> {
  static constexpr uint32_t kOne = 0x39803980u;  // 2^-12
  static constexpr float kOffset = 16.0f, kUnit = 0x1p12f;  // what it has above v; the factor back
  uint32_t sixteen = keep(0x3B803B80u);  // 2^-12 x 16
  __device__ __forceinline__ v4u operator()(uint32_t w) const {
    constexpr uint32_t mask = 0x00780078u;
    return v4u{((w << 3) & mask) | sixteen, ((w >> 1) & mask) | sixteen,
               ((w >> 5) & mask) | sixteen, ((w >> 9) & mask) | sixteen};
  }
};
template <>
struct Unpack<false> {
  static constexpr uint32_t kOne = 0x3C003C00u;
  static constexpr float kOffset = 0.0f, kUnit = 1.0f;
  // 0x6400 | v is 1024 + v and 0x5400 | v << 4 is 64 + v, exactly
  uint32_t big = keep(0x64006400u), mid = keep(0x54005400u);
  __device__ __forceinline__ v4u operator()(uint32_t w) const {
    constexpr uint32_t low = 0x000F000Fu, high = 0x00F000F0u;
    const uint32_t w8 = w >> 8;
    return v4u{less((w & low) | big, big), less((w & high) | mid, mid),
               less((w8 & low) | big, big), less((w8 & high) | mid, mid)};
  }
  static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) - __builtin_bit_cast(v2h, b));
  }
};

template <bool BF>
__device__ __forceinline__ v4f mfma(v4u x, v4u w, v4f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x),
                                                   __builtin_bit_cast(v8bf, w), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x),
                                                  __builtin_bit_cast(v8h, w), c, 0, 0, 0);
}

// A lane's S scales (or zeros) of a record, and the i-th of them.
template <int S>
struct Scales {
  uint32_t u[S == 4 ? 2 : 1];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    if constexpr (S == 4) {
      const uint2 v =
          __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, lane_at, at, 0));
      u[0] = v.x;
      u[1] = v.y;
    } else if constexpr (S == 2) {
      u[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, lane_at, at, 0);
    } else {
      u[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, lane_at, at, 0);
    }
  }
  template <bool BF>
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = u[i >> 1];
    if constexpr (BF)
      return __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
    else
      return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
  }
};

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

// XT: the tokens' type. Q: groups of four tokens: column tiles for float32, else result registers. S:
// scales of a row in a record. SBF: bf16 scales. ALL: x is in LDS for all records of a wavefront, else for
// one, brought in anew for every record of every tile. The sums of `batch` tiles are added together.
template <int XT, int Q, int S, bool SBF, bool ALL>
__global__ __launch_bounds__(64 * max_waves(XT, Q)) void q4g_kernel(
    const void* __restrict__ x, const uint8_t* __restrict__ rep, void* y, int y_type, int M, int N,
    int K, int zeros, int batch, Q4GEpilogue epi) {
  constexpr bool F32 = XT == kTypeF32;
  constexpr bool BF = XT != kTypeF16;
  constexpr int CT = F32 ? Q : 1;
  constexpr bool PAIRS = F32 && Q == 1;
  constexpr int XA = PAIRS ? 2 : 1;  // records whose x is in flight, in registers
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, threads = (int)blockDim.x;
  const int nw = threads >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane >> 4, l16 = lane & 15;
  const int ntiles = (N + kG4Rows - 1) / kG4Rows, nrec = (K + kG4Values - 1) / kG4Values;
  // records of this wavefront in a tile
  const int rounds = wave < nrec ? (nrec - wave + nw - 1) / nw : 0;
  const int slots = ALL ? (nrec + nw - 1) / nw : 1;
  const int rec_bytes = kG4ValueBytes + 32 * S * (zeros ? 2 : 1);
  const uint32_t tile_bytes = (uint32_t)nrec * (uint32_t)rec_bytes;
  const int grid = (int)gridDim.x;

  struct Weights {
    v4i v;
    Scales<S> s, z;
  };
  // record wave + j * nw of a tile
  auto load_w = [&](Weights& r, int tile, int j) {
    if (tile >= ntiles || j >= rounds) return;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(rep + (size_t)tile * tile_bytes, tile_bytes);
    const int o = (wave + j * nw) * rec_bytes;
    r.v = load16(rw, lane * 16, o);
    r.s.load(rw, kG4ValueBytes + l16 * (2 * S), o);
    if (zeros) r.z.load(rw, kG4ValueBytes + 32 * S + l16 * (2 * S), o);
  };

  // x of such a record, as the operands in this wavefront's LDS. Only it uses them, and its LDS operations
  // are in order. 0 past K, where the operand of the weights need not be 0.
  const int rows = x_rows(XT, M), row_bytes = rows * kRowBytes;
  uint8_t* xw = smem + wave * (slots * row_bytes);
  // 16-bit tokens go there by themselves, four tokens to an instruction: lane (c, l16) has the place l16 of
  // token 4 q + c.
  const uint32_t x_bytes = (uint32_t)M * (uint32_t)K * (F32 ? 4u : 2u);
  const v4i rx = make_rsrc_sgpr(x, x_bytes);
  const __amdgpu_buffer_rsrc_t rxb = make_rsrc(x, x_bytes);
  const uint32_t xw_at = lds_addr(smem) + (uint32_t)(wave * (slots * row_bytes));
  auto fetch_x = [&](int j, int slot) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int t = 4 * q + c, k = (wave + j * nw) * kG4Values + 8 * (l16 ^ (t & 15));
      if (t < M)
        dma16(rx, xw_at + (uint32_t)(slot * row_bytes + q * 4 * kRowBytes),
              k < K ? ((uint32_t)t * (uint32_t)K + k) * 2u : x_bytes);
    }
  };
  // float32 tokens through registers: up to four tokens two values of each to a lane, else 16 lanes to a
  // token and eight values to a lane.
  struct Tokens {
    v4u a[PAIRS ? 1 : Q], b[PAIRS ? 1 : Q];
    float2 f[PAIRS ? 4 : 1];
  };
  auto load_x = [&](Tokens& r, int j) {
    if (j >= rounds) return;
    if constexpr (PAIRS) {
      const int k = (wave + j * nw) * kG4Values + 2 * lane;
      const uint32_t at = k < K ? (uint32_t)k * 4u : x_bytes;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < M) r.f[t] = buf_load_f32x2(rxb, at + (uint32_t)t * (uint32_t)K * 4u);
    } else {
      const int k = (wave + j * nw) * kG4Values + 8 * l16;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int t = 4 * q + c;
        const uint32_t at = t < M && k < K ? ((uint32_t)t * (uint32_t)K + k) * 4u : x_bytes;
        r.a[q] = __builtin_bit_cast(v4u, buf_load16(rxb, at));
        r.b[q] = __builtin_bit_cast(v4u, buf_load16(rxb, at + 16));
      }
    }
  };
  auto put_x = [&](const Tokens& r, int slot) {
    uint8_t* xj = xw + slot * row_bytes;
    if constexpr (PAIRS) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= M) break;
        uint32_t a[3], b[3];
        bf16_trunc3(r.f[t].x, a[0], a[1], a[2]);
        bf16_trunc3(r.f[t].y, b[0], b[1], b[2]);
#pragma unroll
        for (int n = 0; n < 3; ++n)
          *reinterpret_cast<uint32_t*>(xj + x_place(3 * t + n, lane >> 2) + (lane & 3) * 4) =
              pack_hi16(a[n], b[n]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int t = 4 * q + c;
        if (t >= M) continue;
        uint32_t pc[8][3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t bits = e < 4 ? r.a[q][e & 3] : r.b[q][e & 3];
          bf16_trunc3(__builtin_bit_cast(float, bits), pc[e][0], pc[e][1], pc[e][2]);
        }
#pragma unroll
        for (int n = 0; n < 3; ++n)
          *reinterpret_cast<v4u*>(xj + x_place(3 * t + n, l16)) =
              v4u{pack_hi16(pc[0][n], pc[1][n]), pack_hi16(pc[2][n], pc[3][n]),
                  pack_hi16(pc[4][n], pc[5][n]), pack_hi16(pc[6][n], pc[7][n])};
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  // This lane's column: of a 16-bit token, or a piece of a float32 one (the fourth column of a token
  // repeats the third). Columns without a token read one that is there; their sums are not used.
  int place[CT][4];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int t = min(F32 ? 4 * ct + (l16 >> 2) : (l16 >> 2) + 4 * (l16 & 3), M - 1);
#pragma unroll
    for (int m = 0; m < 4; ++m) place[ct][m] = x_place(F32 ? 3 * t + min(l16 & 3, 2) : t, 4 * m + c);
  }

  float out[Q];
  const Unpack<BF> unpack;
  constexpr uint32_t one = Unpack<BF>::kOne;
  const v4u ones = v4u{keep(one), keep(one), keep(one), keep(one)};

  auto compute = [&](const Weights& r, const uint8_t* xj) {
    v4f acc[CT], xs[CT];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const v4u wv = unpack((uint32_t)r.v[m]);
      const bool first = m % (4 / S) == 0, last = m % (4 / S) == 4 / S - 1;
      const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const v4u xv = *reinterpret_cast<const v4u*>(xj + place[ct][m]);
        acc[ct] = mfma<BF>(xv, wv, first ? zero : acc[ct]);
        xs[ct] = mfma<BF>(xv, ones, first ? zero : xs[ct]);
      }
      if (last) {
        const int g = m / (4 / S);
        const float sc = r.s.template get<SBF>(g);
        const float z = Unpack<BF>::kOffset + (zeros ? r.z.template get<SBF>(g) : 8.0f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          float a, b;
          if constexpr (F32) {
            a = (acc[q][2] + acc[q][1]) + acc[q][0];
            b = (xs[q][2] + xs[q][1]) + xs[q][0];
          } else {
            a = acc[0][q];
            b = xs[0][q];
          }
          out[q] = __builtin_fmaf(sc, __builtin_fmaf(-z, b, a), out[q]);
        }
      }
    }
  };

  // The wavefronts' sums, [tile of the batch][wave][q][c][row]: lane (c, row) has token c + 4 q.
  float* red = reinterpret_cast<float*>(smem + nw * (slots * row_bytes));
  constexpr int kSums = Q * 64;
  Weights w[kAhead];
  Tokens xr[F32 ? XA : 1];
  if constexpr (ALL && !F32) {
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) fetch_x(j, j);
  }
  if constexpr (F32) {
#pragma unroll
    for (int u = 0; u < XA; ++u) load_x(xr[u], u);
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(w[u], (int)blockIdx.x, u);
  if constexpr (ALL && F32) {
#pragma unroll 1
    for (int j = 0; j < rounds; j += XA) {
#pragma unroll
      for (int u = 0; u < XA; ++u) {
        if (j + u >= rounds) break;
        put_x(xr[u], j + u);
        load_x(xr[u], j + u + XA);
      }
    }
  }
  if constexpr (ALL && !F32) {
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  for (int tile0 = blockIdx.x; tile0 < ntiles; tile0 += batch * grid) {
    int n = 0;
    for (; n < batch; ++n) {
      const int tile = tile0 + n * grid;
      if (tile >= ntiles) break;
#pragma unroll
      for (int q = 0; q < Q; ++q) out[q] = 0.0f;
      for (int j0 = 0; j0 < rounds; j0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int j = j0 + u;
          if (j >= rounds) break;
          if constexpr (!ALL && F32) {
            put_x(xr[u % XA], 0);
            load_x(xr[u % XA], j + XA < rounds ? j + XA : u % XA);
          }
          if constexpr (!ALL && !F32) {
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the last record's operands have been read
            fetch_x(j, 0);
            __builtin_amdgcn_s_waitcnt(0);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
          }
          compute(w[u], xw + (ALL ? j : 0) * row_bytes);
          if (j + kAhead < rounds) load_w(w[u], tile, j + kAhead);
          else load_w(w[u], tile + grid, u);
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) red[(n * nw + wave) * kSums + q * 64 + lane] = out[q];
    }
    __syncthreads();
    for (int i = tid; i < n * kSums; i += threads) {
      const int b = i / kSums, e = i - b * kSums;
      const int t = ((e >> 4) & 3) + 4 * (e >> 6);
      const int j = (tile0 + b * grid) * kG4Rows + (e & 15);
      if (t >= M || j >= N) continue;
      const float* r = red + b * nw * kSums + e;
      float v = r[0];
      for (int k = 1; k < nw; ++k) v += r[k * kSums];
      v *= Unpack<BF>::kUnit;
      if (epi.bias) v += epi.bias[j];
      v = activate(v, epi.act);
      const size_t at = (size_t)t * N + j;
      if (epi.residual) v += load_as_float(epi.residual, at, y_type);
      store_float(y, at, y_type, v);
    }
    if (tile0 + batch * grid < ntiles) __syncthreads();  // the sums have been read
  }
}

// Groups of four tokens that a kernel is built for.
constexpr int token_groups(int64_t M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

// How a call is laid out: wavefronts of a workgroup, records of each that x is in LDS for, tiles whose sums
// are added together, workgroups, and the LDS.
struct Plan {
  int64_t nw, slots, batch, grid, lds;
  bool all;
};
Plan plan(int x_type, int64_t M, const Q4GShape& g, int64_t cus) {
  constexpr int64_t kLds = 160 << 10;
  Plan p;
  const int q = token_groups(M);
  // 8 wavefronts instead of 16 where half of the compute units or fewer have a tile (graph replays, 8 against
  // 16: 1 x 1024 x 4096 f16 4.6 and 4.8 us, 3 x 1376 x 4096 bf16 4.7 and 5.0, 1 x 2048 x 4096 4.8 and 4.9, but
  // 1 x 3000 x 4096 5.0 and 4.9, 1 x 4096 x 4096 5.3 and 5.1), and, as two workgroups to a unit, where every
  // unit has several tiles and a tile's sums are few (1 x 8192 x 4096 7.0 and 7.1, 1 x 11008 x 4096 8.5 and
  // 8.8, 1 x 22016 x 4096 13.1 and 13.4; float32 9.8 and 9.4, 9 tokens 10.0 and 9.8).
  const bool several = g.tiles() >= 2 * cus && q == 1 && x_type != kTypeF32;
  const int64_t per = several ? 2 : 1;
  p.nw = several || 2 * g.tiles() <= cus ? 8 : max_waves(x_type, q);
  while (p.nw > 1 && p.nw > g.records()) p.nw /= 2;
  p.grid = std::min(g.tiles(), per * cus);
  const int64_t row = p.nw * x_rows(x_type, M) * kRowBytes, sums = p.nw * q * 256;
  p.slots = (g.records() + p.nw - 1) / p.nw;
  // one tile: float32 values on their way into LDS between the records, not all before the first
  // (1 x 4096 x 11008 11.1 us against 11.8, 1 x 4096 x 4096
  // 5.0 against 5.6)
  p.all = p.slots * row + sums <= kLds / per && (x_type != kTypeF32 || g.tiles() > cus);
  if (!p.all) p.slots = 1;
  const int64_t most = (g.tiles() + p.grid - 1) / p.grid;
  p.batch = std::max<int64_t>(1, std::min(most, (kLds / per - p.slots * row) / sums));
  p.lds = p.slots * row + p.batch * sums;
  return p;
}

struct Call {
  const void* x;
  const uint8_t* rep;
  void* y;
  int y_type;
  int64_t M;
  Plan p;
  Q4GShape g;
  Q4GEpilogue epi;
};

template <int XT, int Q, int S, bool SBF, bool ALL>
hipError_t launch_k(const Call& c, hipStream_t s) {
  auto kern = q4g_kernel<XT, Q, S, SBF, ALL>;
  if (c.p.lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)c.p.lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)c.p.grid), dim3((unsigned)(64 * c.p.nw)), (size_t)c.p.lds, s,
                     c.x, c.rep, c.y, c.y_type, (int)c.M, (int)c.g.N, (int)c.g.K, (int)c.g.zeros,
                     (int)c.p.batch, c.epi);
  return hipGetLastError();
}

template <int XT, int Q, int S, bool SBF>
hipError_t launch_t(const Call& c, hipStream_t s) {
  return c.p.all ? launch_k<XT, Q, S, SBF, true>(c, s) : launch_k<XT, Q, S, SBF, false>(c, s);
}

template <int XT, int Q>
hipError_t launch_q(const Call& c, bool sbf, hipStream_t s) {
  switch (c.g.scales()) {
    case 1: return sbf ? launch_t<XT, Q, 1, true>(c, s) : launch_t<XT, Q, 1, false>(c, s);
    case 2: return sbf ? launch_t<XT, Q, 2, true>(c, s) : launch_t<XT, Q, 2, false>(c, s);
    default: return sbf ? launch_t<XT, Q, 4, true>(c, s) : launch_t<XT, Q, 4, false>(c, s);
  }
}

template <int XT>
hipError_t launch_x(const Call& c, bool sbf, hipStream_t s) {
  switch (token_groups(c.M)) {
    case 1: return launch_q<XT, 1>(c, sbf, s);
    case 2: return launch_q<XT, 2>(c, sbf, s);
    default: return launch_q<XT, 4>(c, sbf, s);
  }
}

// One work-item per dword of the values, and one per scale and zero, of a record.
__global__ __launch_bounds__(256) void repack_kernel(const uint8_t* __restrict__ w,
                                                     const uint16_t* __restrict__ scales,
                                                     const uint16_t* __restrict__ zeros,
                                                     uint8_t* __restrict__ rep, int64_t N, int64_t K,
                                                     int64_t group, int64_t nrec, int64_t ngroups,
                                                     int S, int rec_bytes) {
  const int64_t tile = (int64_t)blockIdx.x / nrec, rec = (int64_t)blockIdx.x - tile * nrec;
  uint8_t* out = rep + (int64_t)blockIdx.x * rec_bytes;
  const int q = threadIdx.x;
  {
    const int m = q & 3, row = (q >> 2) & 15, c = q >> 6;
    const int64_t j = tile * kG4Rows + row, k = rec * kG4Values + 32 * m + 8 * c;
    uint32_t o = 0;
    if (j < N && k < K) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(w + (j * K + k) / 2);
      // nibble e of v (value e) goes to nibble e / 2 + 4 (e % 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) o |= ((v >> (4 * e)) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
    }
    reinterpret_cast<uint32_t*>(out)[q] = o;
  }
  const int n = kG4Rows * S;
  if (q < (zeros ? 2 * n : n)) {
    const uint16_t* src = q < n ? scales : zeros;
    const int i = q < n ? q : q - n;
    const int64_t j = tile * kG4Rows + i / S;
    const int64_t k = rec * kG4Values + (i % S) * (kG4Values / S);
    reinterpret_cast<uint16_t*>(out + kG4ValueBytes)[q] =
        j < N && k < K ? src[j * ngroups + k / group] : (uint16_t)0;
  }
}

}  // namespace

int64_t q4g_lds_bytes(int x_type, int64_t M, const Q4GShape& g, int64_t compute_units) {
  return plan(x_type, M, g, compute_units).lds;
}

hipError_t launch_q4g(const void* x, int x_type, const void* rep, int scale_type, void* y,
                      int y_type, int64_t M, const Q4GShape& g, const Q4GEpilogue& epi,
                      int64_t compute_units, hipStream_t s) {
  const Call c{x, static_cast<const uint8_t*>(rep), y, y_type, M, plan(x_type, M, g, compute_units), g,
               epi};
  const bool sbf = scale_type == kTypeBF16;
  return x_type == kTypeF32   ? launch_x<kTypeF32>(c, sbf, s)
         : x_type == kTypeF16 ? launch_x<kTypeF16>(c, sbf, s)
                              : launch_x<kTypeBF16>(c, sbf, s);
}

hipError_t launch_repack_q4g(const void* w, const void* scales, const void* zeros,
                             const Q4GShape& g, void* rep, hipStream_t s) {
  static_assert(2 * kG4Rows * 4 <= 256, "a work-item per scale and zero");
  hipLaunchKernelGGL(repack_kernel, dim3((unsigned)(g.tiles() * g.records())), dim3(256), 0, s,
                     static_cast<const uint8_t*>(w), static_cast<const uint16_t*>(scales),
                     static_cast<const uint16_t*>(zeros), static_cast<uint8_t*>(rep), g.N, g.K,
                     g.group, g.records(), g.groups(), g.scales(), (int)g.record_bytes());
  return hipGetLastError();
}

}  // namespace mmq
