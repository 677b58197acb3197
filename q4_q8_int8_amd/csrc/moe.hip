// The two products of a mixture-of-experts layer for a few tokens, over q4_K weights and q8_1
// activations (the arithmetic of the GEMM, mmq_gemm.hip), reading each used expert once.
//
// With p = t * k + s the pair (token t, slot s), e(p) its expert and a(p) its activations:
//   gated   H[p] = act(x[t] Wg(e)^T) * (x[t] Wu(e)^T)        (pair records, epilogue.h)
//   down    out[t] = sum over the slots s of weight[p] * (H[p] Wd(e)^T) + residual[t]
// The plan (moe_route.hip) lists the used experts in increasing order, each with its pairs, so a
// workgroup of an expert finds the rows of its product, the expert's columns below, in one list.
//
// Both are bound by reading the used experts' weights: with few tokens an expert has a handful of
// columns, the weights are 4.5 bits each, and nothing else is of their size. One matrix
// instruction, v_mfma_i32_16x16x32_i8, takes one 32-block of 16 weight rows against 16 columns,
// so up to 16 columns cost what one does, and the kernels are the decode tile's matrix-unit form
// (mmq_gemv.hip) with the columns gathered: 16-byte pieces of any row of q8 go to the
// wavefront's own LDS region by direct-to-LDS loads. Columns past the expert's are never loaded:
// what LDS holds in their place only reaches result columns that nobody stores.
//
// Per super-block of 256 k a wavefront does
//   D   = MFMA_i8(w, q, bias)          one per block and 16 rows, S exactly
//   y   = fma(D, da, -1.5*2^23*da)     RN(S * da)
//   acc = fma(y, dsv, acc)
// and two bf16 MFMAs add term2 from exact three-piece splits of dmv and da*sa (mmq_gemv.hip).
// Sums are float32 in a fixed order: super-blocks of a wavefront in increasing order, then the
// wavefronts in order. No atomics; the same bits on every call.
#include "epilogue.h"
#include "mmq_device.h"
#include "moe_internal.h"

namespace mmq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// A wavefront's LDS: per 16-row half its expanded scales (dsv f32 [8][16], then the dmv pieces
// bf16 [3][16][8]); its columns' operands of one super-block: int8 [NT][256], the 16-byte chunk c
// of column t at chunk c ^ t, then the da*sa pieces bf16 [3][NT][8].
constexpr int kDsvBytes = 8 * 16 * 4;
constexpr int kScaleBytes = kDsvBytes + 3 * 16 * 8 * 2;
template <int NT>
constexpr int kTokBytes = NT * 256 + 3 * NT * 16;

// Everything a wavefront keeps of a q8 buffer of `rows` x K.
struct Q8 {
  v4i rq, rpc;                    // q, the da*sa pieces (direct-to-LDS descriptors)
  __amdgpu_buffer_rsrc_t rwd;     // the packed (da, sa) words
  uint32_t rows, K, kb;
};
__device__ __forceinline__ Q8 make_q8(const uint8_t* base, int rows, int K) {
  Q8 q;
  q.rows = (uint32_t)rows;
  q.K = (uint32_t)K;
  q.kb = (uint32_t)(K >> 5);
  q.rq = make_rsrc_sgpr(base, q.rows * q.K);
  q.rpc = make_rsrc_sgpr(base + q8_pieces_offset(rows, K), q.rows * (q.K >> 8) * 48u);
  q.rwd = make_rsrc(base + (size_t)rows * K, q.rows * q.kb * 4u);
  return q;
}

// A group of up to NT columns: lane l stages 16-byte chunks of columns 4 i + l / 16 and, below
// 3 NT, piece l / NT of column l % NT; as an operand lane it has column l % 16 (modulo NT).
template <int NT>
struct Columns {
  uint32_t stage_row[NT / 4];  // q8 row of column 4 i + l / 16
  uint32_t piece_row;          // q8 row of column l % NT
  uint32_t row;                // q8 row of column (l % 16) % NT
  int n;                       // columns in use (wave-uniform)
};

template <int NT>
__device__ __forceinline__ void stage_columns(const Q8& q, const Columns<NT>& c, uint32_t tok,
                                              int s, int lane) {
#pragma unroll
  for (int i = 0; i < NT / 4; ++i) {
    if (4 * i < c.n) {  // wave-uniform
      const int t = 4 * i + (lane >> 4), ch = (lane & 15) ^ t;
      dma16(q.rq, tok + i * 1024, c.stage_row[i] * q.K + (uint32_t)s * 256u + (uint32_t)ch * 16u);
    }
  }
  if (lane < 3 * NT)
    dma16(q.rpc, tok + NT * 256,
          (((uint32_t)s * 3u + (uint32_t)(lane / NT)) * q.rows + c.piece_row) * 16u);
}

// The weights of one super-block record for RT halves of its 32 rows, `half0` the first.
template <int RT>
struct Weights {
  uint2 nib[RT][4];
  v4i hdr[RT];
};
template <int RT>
__device__ __forceinline__ void load_weights(__amdgpu_buffer_rsrc_t rw, uint32_t rec, int half0,
                                             int c16, int kg, Weights<RT>& w) {
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    const int j = (half0 + h) * 16 + c16;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      w.nib[h][g] = __builtin_bit_cast(
          uint2, buf_load_f32x2(rw, rec + g * 1024 + (kg >> 1) * 512 + j * 16 + (kg & 1) * 8));
    w.hdr[h] = buf_load16(rw, rec + kRepNibBytes + j * 16);
  }
}

// Lane (c16, kg) expands sub-blocks 2 kg and 2 kg + 1 of row c16 of each half into LDS.
template <int RT>
__device__ __forceinline__ void expand_scales(const Weights<RT>& w, uint8_t* ss, int c16, int kg) {
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    float dsv4[4], dmv4[4];
    q4k_scales(w.hdr[h], kg >= 2, dsv4, dmv4);
    const bool odd = (kg & 1) != 0;
    uint32_t pa[3], pb[3];
    bf16_trunc3(odd ? dmv4[2] : dmv4[0], pa[0], pa[1], pa[2]);
    bf16_trunc3(odd ? dmv4[3] : dmv4[1], pb[0], pb[1], pb[2]);
    float* sd = reinterpret_cast<float*>(ss + h * kScaleBytes);
    sd[(2 * kg) * 16 + c16] = odd ? dsv4[2] : dsv4[0];
    sd[(2 * kg + 1) * 16 + c16] = odd ? dsv4[3] : dsv4[1];
    uint32_t* sp = reinterpret_cast<uint32_t*>(ss + h * kScaleBytes + kDsvBytes);
#pragma unroll
    for (int i = 0; i < 3; ++i) sp[(i * 16 + c16) * 4 + kg] = pack_hi16(pa[i], pb[i]);
  }
}

// acc += one super-block: its weights in w, its scales in ss, its columns in stok (LDS), da[b] the
// column's scale of block b. Result layout: register r of lane (c16, kg) is row 4 kg + r of the
// half and column c16.
template <int RT, int NT>
__device__ __forceinline__ void multiply(const Weights<RT>& w, const uint8_t* ss,
                                         const uint8_t* stok, const float (&da)[8], v4i bias,
                                         int c16, int kg, v4f (&acc)[RT]) {
  const int col = c16 & (NT - 1);
  // term2 piece pairs of this lane's k-group, as in mmq_gemv.hip: (0,0) (0,1) (1,0) (0,2) in the
  // first instruction, (1,1) (2,0) and two zero groups in the second
  const int ia1 = kg == 2 ? 1 : 0, jb1 = kg == 1 ? 1 : (kg == 3 ? 2 : 0);
  const int ia2 = kg == 1 ? 2 : 1, jb2 = kg == 0 ? 1 : 0;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint2 tb = *reinterpret_cast<const uint2*>(
        stok + col * 256 + (((2 * b + (kg >> 1)) ^ col) << 4) + (kg & 1) * 8);
    const float nda = -kBiasF * da[b];
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      const uint2 n = w.nib[h][b >> 1];
      const uint2 a = (b & 1) ? make_uint2((n.x >> 4) & 0x0F0F0F0Fu, (n.y >> 4) & 0x0F0F0F0Fu)
                              : make_uint2(n.x & 0x0F0F0F0Fu, n.y & 0x0F0F0F0Fu);
      const v4i D = __builtin_amdgcn_mfma_i32_16x16x32_i8(
          __builtin_bit_cast(long, a), __builtin_bit_cast(long, tb), bias, 0, 0, 0);
      const float4 dq = *reinterpret_cast<const float4*>(ss + h * kScaleBytes + (b * 16 + 4 * kg) * 4);
      const float dsv[4] = {dq.x, dq.y, dq.z, dq.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float y = __builtin_fmaf(__int_as_float(D[r]), da[b], nda);
        acc[h][r] = __builtin_fmaf(y, dsv[r], acc[h][r]);
      }
    }
  }
  const uint8_t* pc = stok + NT * 256;
  const v4i pb0 = *reinterpret_cast<const v4i*>(pc + (jb1 * NT + col) * 16);
  const v4i pb1 = *reinterpret_cast<const v4i*>(pc + (jb2 * NT + col) * 16);
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    const uint8_t* sp = ss + h * kScaleBytes + kDsvBytes;
    const v4i pa0 = *reinterpret_cast<const v4i*>(sp + (ia1 * 16 + c16) * 16);
    v4i pa1 = *reinterpret_cast<const v4i*>(sp + (ia2 * 16 + c16) * 16);
    if (kg >= 2) pa1 = v4i{0, 0, 0, 0};
    acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, pa0),
                                                     __builtin_bit_cast(v8bf, pb0), acc[h], 0, 0, 0);
    acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, pa1),
                                                     __builtin_bit_cast(v8bf, pb1), acc[h], 0, 0, 0);
  }
}

// The column's eight scales da of super-block s, from the packed (da, sa) words of its row.
__device__ __forceinline__ void load_words(const Q8& q, uint32_t row, int s, v4i (&wd)[2]) {
  const uint32_t at = (row * q.kb + (uint32_t)s * 8u) * 4u;
  wd[0] = buf_load16(q.rwd, at);
  wd[1] = buf_load16(q.rwd, at + 16u);
}
__device__ __forceinline__ void unpack_da(const v4i (&wd)[2], float (&da)[8]) {
#pragma unroll
  for (int b = 0; b < 8; ++b)
    da[b] = (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)wd[b >> 2][b & 3] & 0xFFFFu));
}

// Wavefront-wide ordering of its own LDS region and its direct-to-LDS loads: everything issued
// has arrived (vmcnt 0, lgkmcnt 0) and later reads stay below.
__device__ __forceinline__ void wave_sync_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Pair p of position i of an expert's list, kept inside the buffers whatever the plan holds.
__device__ __forceinline__ int pair_at(const int* order, int i, int P) {
  const int p = order[i];
  return p < 0 ? 0 : (p < P ? p : P - 1);
}

// ---------------------------------------------------------------- the gated product

// Workgroup (u, tile): used expert u, one 32-row tile of its pair records (16 columns of H), all
// of K: wavefront w takes the super-blocks w, w + NW, ....
template <int NW, int NT>
__global__ __launch_bounds__(64 * NW) void moe_gated_kernel(
    const uint8_t* __restrict__ q8, const int* __restrict__ plan, const uint8_t* __restrict__ wrep,
    float* __restrict__ H, int M, int E, int k, int F, int K, int entries, int act) {
  constexpr int RT = 2;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kTokOff = NW * RT * kScaleBytes;
  constexpr int kRedOff = kTokOff + NW * kTokBytes<NT>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int c16 = lane & 15, kg = lane >> 4;
  const int tiles = (F + 15) >> 4;
  const int u = (int)(blockIdx.x / (unsigned)tiles), tile = (int)(blockIdx.x % (unsigned)tiles);
  const int P = M * k;
  const PlanEntry en = plan_entry(plan, u, E, P);
  if (en.n == 0) return;
  const int* order = plan + kPlanHead + 4 * entries + en.first;
  const int nsb = K >> 8;
  const uint8_t* wtile = wrep + ((size_t)en.expert * tiles + tile) * (size_t)nsb * kRepTileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wtile, (uint32_t)nsb * (uint32_t)kRepTileBytes);
  const Q8 q = make_q8(q8, M, K);
  uint8_t* ss = smem + wave * RT * kScaleBytes;
  const uint8_t* stok = smem + kTokOff + wave * kTokBytes<NT>;
  const uint32_t tok = lds_addr(smem) + (uint32_t)(kTokOff + wave * kTokBytes<NT>);
  float* red = reinterpret_cast<float*>(smem + kRedOff);  // [NW][NT][32]
  v4i bias = {kBiasBits, kBiasBits, kBiasBits, kBiasBits};
  asm volatile("" : "+v"(bias));

  for (int g0 = 0; g0 < en.n; g0 += NT) {
    Columns<NT> c;
    c.n = en.n - g0 < NT ? en.n - g0 : NT;
    auto token_of = [&](int t) {
      return (uint32_t)(pair_at(order, g0 + (t < c.n ? t : c.n - 1), P) / k);
    };
#pragma unroll
    for (int i = 0; i < NT / 4; ++i) c.stage_row[i] = token_of(4 * i + (lane >> 4));
    c.piece_row = token_of(lane % NT);
    c.row = token_of(c16 & (NT - 1));
    v4f acc[RT];
#pragma unroll
    for (int h = 0; h < RT; ++h) acc[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = wave; s < nsb; s += NW) {
      Weights<RT> w;
      v4i wd[2];
      float da[8];
      load_weights<RT>(rw, (uint32_t)s * kRepTileBytes, 0, c16, kg, w);
      load_words(q, c.row, s, wd);
      stage_columns<NT>(q, c, tok, s, lane);
      expand_scales<RT>(w, ss, c16, kg);
      wave_sync_all();
      unpack_da(wd, da);
      multiply<RT, NT>(w, ss, stok, da, bias, c16, kg, acc);
      wave_sync_all();  // the region is read: the next super-block may overwrite it
    }
    if (c16 < NT) {
#pragma unroll
      for (int h = 0; h < RT; ++h)
        *reinterpret_cast<v4f*>(red + (wave * NT + c16) * 32 + h * 16 + 4 * kg) = acc[h];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < NT * 16; e += 64 * NW) {
      const int t = e >> 4, fl = e & 15;
      const int f = tile * 16 + fl, gr = 16 * (fl >> 3) + (fl & 7);
      if (t < c.n && f < F) {
        float g = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          g += red[(w * NT + t) * 32 + gr];
          v += red[(w * NT + t) * 32 + gr + 8];
        }
        H[(size_t)pair_at(order, g0 + t, P) * F + f] = activate(g, act) * v;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the down product

// Workgroup: 16 rows of N (half a tile), every used expert. Its wavefronts deal the
// (expert, super-block) items among them and each adds weight * acc of an item's columns to its
// own sums [M][16] in LDS; at the end the wavefronts' sums are added in order. So the sum over
// the slots needs no memory, no atomics and no second launch.
template <int NW, int NT>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(
    const uint8_t* __restrict__ q8, const int* __restrict__ plan,
    const float* __restrict__ weights, const uint8_t* __restrict__ wrep,
    const float* residual, float* out, int M, int E, int k, int N, int K, int entries) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kTokOff = NW * kScaleBytes;
  constexpr int kRedOff = kTokOff + NW * kTokBytes<NT>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int c16 = lane & 15, kg = lane >> 4;
  const int rb = (int)blockIdx.x;
  const int P = M * k;
  const int nsb = K >> 8;
  const int tiles = (N + 31) >> 5;
  const Q8 q = make_q8(q8, P, K);
  uint8_t* ss = smem + wave * kScaleBytes;
  const uint8_t* stok = smem + kTokOff + wave * kTokBytes<NT>;
  const uint32_t tok = lds_addr(smem) + (uint32_t)(kTokOff + wave * kTokBytes<NT>);
  float* sums = reinterpret_cast<float*>(smem + kRedOff) + wave * M * 16;  // [M][16]
  v4i bias = {kBiasBits, kBiasBits, kBiasBits, kBiasBits};
  asm volatile("" : "+v"(bias));
  for (int i = lane; i < M * 16; i += 64) sums[i] = 0.0f;

  int used = plan[0];
  if (used < 0 || used > entries) used = 0;
  const int* lists = plan + kPlanHead + 4 * entries;
  for (int item = wave; item < used * nsb; item += NW) {  // at most 512 x 2^16 items
    const int u = item / nsb, s = item - u * nsb;
    const PlanEntry en = plan_entry(plan, u, E, P);
    if (en.n == 0) continue;
    const int* order = lists + en.first;
    const uint8_t* wtile =
        wrep + ((size_t)en.expert * tiles + (rb >> 1)) * (size_t)nsb * kRepTileBytes;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(wtile, (uint32_t)nsb * (uint32_t)kRepTileBytes);
    Weights<1> w;
    load_weights<1>(rw, (uint32_t)s * kRepTileBytes, rb & 1, c16, kg, w);
    expand_scales<1>(w, ss, c16, kg);
    for (int g0 = 0; g0 < en.n; g0 += NT) {
      Columns<NT> c;
      c.n = en.n - g0 < NT ? en.n - g0 : NT;
      auto pair_of = [&](int t) {
        return pair_at(order, g0 + (t < c.n ? t : c.n - 1), P);
      };
#pragma unroll
      for (int i = 0; i < NT / 4; ++i) c.stage_row[i] = (uint32_t)pair_of(4 * i + (lane >> 4));
      c.piece_row = (uint32_t)pair_of(lane % NT);
      const int p = pair_of(c16 & (NT - 1));
      c.row = (uint32_t)p;
      v4i wd[2];
      float da[8];
      load_words(q, c.row, s, wd);
      const float wt = weights[p];
      stage_columns<NT>(q, c, tok, s, lane);
      wave_sync_all();
      unpack_da(wd, da);
      v4f acc[1] = {v4f{0.0f, 0.0f, 0.0f, 0.0f}};
      multiply<1, NT>(w, ss, stok, da, bias, c16, kg, acc);
      // Columns of one token (an expert named twice by it) are neighbours in the list: they take
      // turns, each turn adding at most one column per token.
      const int t = p / k;
      const int before = __shfl_up(t, 1, 16);
      const bool mine = c16 < c.n;
      uint64_t same = __ballot(mine && c16 > 0 && before == t) & 0xFFFFu;
      int turn = 0;
      if (same) {  // how many of the columns just before this one have its token
        uint32_t m = (uint32_t)same;
        for (int b = c16; b > 0 && ((m >> b) & 1u); --b) ++turn;
      }
      for (int r = 0;; ++r) {
        if (mine && turn == r) {
          v4f* to = reinterpret_cast<v4f*>(sums + t * 16 + 4 * kg);
          v4f v = *to;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(wt, acc[0][i], v[i]);
          *to = v;
        }
        if (!__ballot(mine && turn > r)) break;
        wave_sync_all();
      }
      wave_sync_all();  // the region is read: the next group may overwrite it
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + kRedOff);
  for (int e = threadIdx.x; e < M * 16; e += 64 * NW) {
    const int t = e >> 4, n = rb * 16 + (e & 15);
    if (n < N) {
      float v = 0.0f;
      for (int w = 0; w < NW; ++w) v += all[w * M * 16 + e];
      const size_t at = (size_t)t * N + n;
      out[at] = residual ? v + residual[at] : v;
    }
  }
}

template <int NW, int NT>
int64_t gated_lds() {
  return NW * (2 * kScaleBytes + kTokBytes<NT> + NT * 32 * 4);
}
template <int NW, int NT>
int64_t down_lds(int64_t M) {
  return NW * (kScaleBytes + kTokBytes<NT> + M * 16 * 4);
}

template <int NW, int NT>
hipError_t launch_gated(const void* q8, const int* plan, const void* w, float* H, const MoeShape& m,
                        int act, hipStream_t s) {
  auto kern = moe_gated_kernel<NW, NT>;
  const int64_t lds = gated_lds<NW, NT>();
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const int64_t grid = m.entries() * ((m.F + 15) / 16);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * NW), (size_t)lds, s,
                     static_cast<const uint8_t*>(q8), plan, static_cast<const uint8_t*>(w), H,
                     (int)m.M, (int)m.E, (int)m.k, (int)m.F, (int)m.D, (int)m.entries(), act);
  return hipGetLastError();
}

template <int NW, int NT>
hipError_t launch_down(const void* q8, const int* plan, const float* weights, const void* w,
                       const float* residual, float* out, const MoeShape& m, hipStream_t s) {
  auto kern = moe_down_kernel<NW, NT>;
  const int64_t lds = down_lds<NW, NT>(m.M);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)((m.D + 15) / 16)), dim3(64 * NW), (size_t)lds, s,
                     static_cast<const uint8_t*>(q8), plan, weights,
                     static_cast<const uint8_t*>(w), residual, out, (int)m.M, (int)m.E, (int)m.k,
                     (int)m.D, (int)m.F, (int)m.entries());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_gated(const void* q8, const int* plan, const void* w, float* H,
                            const MoeShape& m, int act, hipStream_t s) {
  return m.M <= 4 ? launch_gated<8, 4>(q8, plan, w, H, m, act, s)
                  : launch_gated<8, 16>(q8, plan, w, H, m, act, s);
}

hipError_t launch_moe_down(const void* q8, const int* plan, const float* weights, const void* w,
                           const float* residual, float* out, const MoeShape& m, hipStream_t s) {
  return m.M <= 4 ? launch_down<16, 4>(q8, plan, weights, w, residual, out, m, s)
                  : launch_down<8, 16>(q8, plan, weights, w, residual, out, m, s);
}

int64_t moe_lds_bytes(int64_t M) {
  const int64_t g = M <= 4 ? gated_lds<8, 4>() : gated_lds<8, 16>();
  const int64_t d = M <= 4 ? down_lds<16, 4>(M) : down_lds<8, 16>(M);
  return g > d ? g : d;
}

}  // namespace mmq
