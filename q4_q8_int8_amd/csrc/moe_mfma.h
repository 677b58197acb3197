// The matrix-unit form of the experts' products (not part of the ABI): up to 16 columns against 16
// or 32 weight rows of one expert per wavefront, one v_mfma_i32_16x16x32_i8 per 32-block and 16
// rows. The columns are gathered: 16-byte pieces of any row of q8 go to the wavefront's LDS by
// direct-to-LDS loads. Columns past the expert's are never loaded: what LDS holds in their place
// only reaches result columns that nobody takes.
//
// Per super-block (a step):
//   D   = MFMA_i8(w, q, bias)          S exactly, biased by 1.5*2^23
//   y   = fma(D, da, -1.5*2^23*da)     RN(S * da)
//   acc = fma(y, dsv, acc)             term1 of a block
//   acc = MFMA_f32(dmv, da*sa, acc)    term2 of all 8 blocks, two v_mfma_f32_16x16x4_f32
// dmv = -dmin*m and da*sa are exact in float32 (17 and 23 significant bits), so term2's products
// are rounded once into the float32 sum, as term1's are. (The large products take term2 to the
// bf16 unit in exact pieces, which is faster there; here the f32 instruction has time to spare,
// and needs no pieces: 40 vector instructions fewer per 32 rows and super-block.)
//
// Up to 16 columns cost what one does, 165 vector instructions per super-block and 16 rows, 64 of
// them the rescale. That bounds the form beside the memory: at 16 tokens, 2 of 8 experts (D = 4096, F =
// 11008) the vector ALU is 63 % busy while the weights come at 4.5 TB/s.
//
// KS = 2: 8 weight rows and two super-blocks at a time. Operand rows 0..7 are the rows of the first
// super-block and 8..15 the same rows of the second, operand columns 0..7 the columns of the first
// and 8..15 of the second; the two diagonal 8 x 8 quarters of the result are the two super-blocks'
// sums, the others are left. An expert of up to 8 columns costs as much per weight as with 16 rows,
// and an output of few rows gives twice the workgroups.
//
// Operand layout: A row and B column l % 16 take the 8 k values 8 (l / 16) .. + 7 (int8), or k =
// l / 16 (f32); register r of lane l is row 4 (l / 16) + r, column l % 16 of the result.
#pragma once

#include "mmq_device.h"
#include "moe_dot.h"

namespace mmq {

typedef float v4f __attribute__((ext_vector_type(4)));

// ONCE: the weights are read once (an expert has no second group of columns, as a rule), and loaded
// so: 16 tokens, 2 of 8 experts, the gated product 96.5 -> 90.2 us; 64 tokens, with experts of more than
// 16 columns, 142 -> 150.
template <int RT, int KS = 1, bool ONCE = false>
struct MfmaWave {
  static_assert(KS == 1 || (KS == 2 && RT == 1), "forms");
  static constexpr int kRows = 16 * RT / KS;
  static constexpr int kCols = 16 / KS;
  static constexpr bool kFused = false;
  static constexpr int SB = KS;
  // LDS: per 16 rows dsv f32 [8][16], then the columns' int8 [16][256], the 16-byte chunk c of
  // column t at chunk c ^ t (every column starts at bank 0: the XOR spreads the operand reads)
  static constexpr int kDsv = 8 * 16 * 4;
  static constexpr int kLds = RT * kDsv + 16 * 256;

  struct Tokens {
    v4i rq;                        // int8 q, for the direct-to-LDS loads
    __amdgpu_buffer_rsrc_t words;  // packed (da, sa)
    uint32_t K, kb;
  };
  static __device__ __forceinline__ Tokens tokens(const void* p, int rows, int K) {
    const uint8_t* base = static_cast<const uint8_t*>(p);
    Tokens t;
    t.K = (uint32_t)K;
    t.kb = (uint32_t)(K >> 5);
    t.rq = make_rsrc_sgpr(base, (uint32_t)rows * t.K);
    t.words = make_rsrc(base + (size_t)rows * K, (uint32_t)rows * t.kb * 4u);
    return t;
  }

  // n columns (wave-uniform). Staged column t is column t % kCols of super-block t / kCols of the
  // step. Lane l stages 16-byte chunks of staged columns 4 i + l / 16; as an operand lane it has
  // staged column l % 16.
  struct Group {
    uint4v drow;                     // q8 row of staged column 4 i + l / 16
    uint32_t row;                    // q8 row of staged column l % 16
    int n, fill0, fill1;             // (no padding: a copy of it would go through scratch memory)
  };
  template <typename RowOf>
  __device__ __forceinline__ Group group(int n, RowOf row_of) const {
    Group g;
    g.n = n;
    g.fill0 = g.fill1 = 0;
    auto at = [&](int t) { return row_of(t % kCols < n ? t % kCols : n - 1); };
#pragma unroll
    for (int i = 0; i < 4; ++i) g.drow[i] = at(4 * i + kg);
    g.row = at(c16);
    return g;
  }

  struct Regs {
    uint2 nib[RT][4];
    v4i hdr[RT];
    v4i wd[2];     // the column's eight (da, sa) words
    float wt[2];   // its words of blocks kg and kg + 4 (bits)
  };
  struct Acc {
    v4f v[RT];
  };

  int lane, c16, kg;
  int row, sel;  // operand row's weight row, and the super-block of the step of row and column
  uint8_t* lds;
  uint32_t lds_at;
  v4i bias;
  float dm[RT][2];  // dmv of the operand row's blocks kg and kg + 4

  __device__ __forceinline__ void init(uint8_t* region, uint32_t at) {
    lane = threadIdx.x & 63;
    c16 = lane & 15;
    kg = lane >> 4;
    row = KS == 2 ? c16 & 7 : c16;
    sel = KS == 2 ? c16 >> 3 : 0;
    lds = region;
    lds_at = at;
    bias = v4i{kBiasBits, kBiasBits, kBiasBits, kBiasBits};
    asm volatile("" : "+v"(bias));
  }

  // Where a step's weights are: rows j0 .. of the tile of `rw`.
  struct Src {
    __amdgpu_buffer_rsrc_t rw;
    uint32_t rec;  // the lane's record; past the end of the tile: nothing is loaded
    int j0, s;     // the step's first super-block
    bool ok;       // the lane's super-block is there
  };
  __device__ __forceinline__ Src source(__amdgpu_buffer_rsrc_t rw, int j0, int nsb, int j,
                                        bool any) const {
    const int s = KS * j + sel;
    const bool ok = any && (KS == 1 || s < nsb);
    return Src{rw, ok ? (uint32_t)s * kRepTileBytes : kNoRecord, j0, KS * j, ok};
  }
  __device__ __forceinline__ void load_weights(const Src& f, Regs& r) const {
    constexpr int AUX = ONCE ? kReadOnce : 0;
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      const int j = f.j0 + h * 16 + row;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.nib[h][i] = buf_load8_aux<AUX>(
            f.rw, f.rec + i * 1024 + (kg >> 1) * 512 + j * 16 + (kg & 1) * 8);
      r.hdr[h] = buf_load16_aux<AUX>(f.rw, f.rec + kRepNibBytes + j * 16);
    }
  }
  __device__ __forceinline__ void load_words(const Tokens& t, const Group& g, int s, bool ok,
                                             Regs& r) const {
    // no super-block: scales of 0
    const uint32_t at = ok ? (g.row * t.kb + (uint32_t)(s + sel) * 8u) * 4u : kNoRecord;
    r.wd[0] = buf_load16(t.words, at);
    r.wd[1] = buf_load16(t.words, at + 16u);
    r.wt[0] = buf_load_f32(t.words, at + 4u * (uint32_t)kg);
    r.wt[1] = buf_load_f32(t.words, at + 4u * (uint32_t)kg + 16u);
  }
  // What of step j's columns is loaded ahead of finish().
  __device__ __forceinline__ void load_columns(const Tokens& t, const Group& g, int j, int nsb,
                                               int, Regs& r) const {
    load_words(t, g, KS * j, KS == 1 || KS * j + sel < nsb, r);
  }

  // Once the previous step is computed: stage the columns, expand the scales of blocks kg and
  // kg + 4 of the operand row (dsv to LDS, dmv to registers), wait.
  __device__ __forceinline__ void finish(const Tokens& t, const Group& g, const Src& f, int,
                                         const Regs& r) {
    asm volatile("" ::: "memory");       // the previous step's LDS reads stay above
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): ... and are done before LDS is written
    const uint32_t tok = lds_at + RT * kDsv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i % kCols < g.n) {  // wave-uniform
        const int c = 4 * i + kg, ch = c16 ^ c;
        dma16(t.rq, tok + i * 1024,
              g.drow[i] * t.K + (uint32_t)(f.s + c / kCols) * 256u + (uint32_t)ch * 16u);
      }
    }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      // sub-block b < 4 has sc = s0[b] & 63 and m = s1[b] & 63; b + 4 has the low four bits of sc
      // and m in the nibbles of s2[b] and their top two bits above the six of s0[b] and s1[b]
      const uint32_t w0 = (uint32_t)r.hdr[h][0];
      const uint32_t s0 = (uint32_t)r.hdr[h][1] >> (8 * kg), s1 = (uint32_t)r.hdr[h][2] >> (8 * kg),
                     s2 = (uint32_t)r.hdr[h][3] >> (8 * kg);
      const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)(w0 & 0xFFFFu));
      const float nm = -(float)__builtin_bit_cast(_Float16, (uint16_t)(w0 >> 16));
      float* sd = reinterpret_cast<float*>(lds + h * kDsv);
      sd[kg * 16 + c16] = d * (float)(s0 & 63u);
      sd[(kg + 4) * 16 + c16] = d * (float)((s2 & 15u) | ((s0 >> 2) & 48u));
      dm[h][0] = nm * (float)(s1 & 63u);
      dm[h][1] = nm * (float)(((s2 >> 4) & 15u) | ((s1 >> 2) & 48u));
    }
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // acc += the step whose registers r are; they are then the next step's (f, columns gn), loaded
  // behind this one's work.
  __device__ __forceinline__ void compute(const Group&, int, int, int, Regs& r, Acc& acc, bool,
                                          const Src& f, const Tokens& t, const Group& gn) const {
    Regs nx;
    load_weights(f, nx);
    load_words(t, gn, f.s, f.ok, nx);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* stok = lds + RT * kDsv + c16 * 256 + (kg & 1) * 8;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint2 tb = *reinterpret_cast<const uint2*>(stok + (((2 * b + (kg >> 1)) ^ c16) << 4));
      const float da = (float)__builtin_bit_cast(
          _Float16, (uint16_t)((uint32_t)r.wd[b >> 2][b & 3] & 0xFFFFu));
      const float nda = -kBiasF * da;
#pragma unroll
      for (int h = 0; h < RT; ++h) {
        const uint2 n = r.nib[h][b >> 1];
        const uint2 a = (b & 1)
                            ? make_uint2((n.x >> 4) & 0x0F0F0F0Fu, (n.y >> 4) & 0x0F0F0F0Fu)
                            : make_uint2(n.x & 0x0F0F0F0Fu, n.y & 0x0F0F0F0Fu);
        const v4i D = __builtin_amdgcn_mfma_i32_16x16x32_i8(
            __builtin_bit_cast(long, a), __builtin_bit_cast(long, tb), bias, 0, 0, 0);
        const v4f dsv = *reinterpret_cast<const v4f*>(lds + h * kDsv + (b * 16 + 4 * kg) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = __builtin_fmaf(__int_as_float(D[i]), da, nda);
          acc.v[h][i] = __builtin_fmaf(y, dsv[i], acc.v[h][i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = __float_as_uint(r.wt[i]);
      const float dma = (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xFFFFu)) *
                        (float)((int)w >> 16);
#pragma unroll
      for (int h = 0; h < RT; ++h)
        acc.v[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(dm[h][i], dma, acc.v[h], 0, 0, 0);
    }
    r = nx;
  }

  static __device__ __forceinline__ void zero(Acc& a) {
#pragma unroll
    for (int h = 0; h < RT; ++h) a.v[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // The finished sums: to(column, first of 4 rows, the 4 values), by the lane that has them.
  template <typename To>
  __device__ __forceinline__ void each(const Group& g, const Acc& a, To to) const {
    if constexpr (KS == 2) {
      v4f v = a.v[0];  // rows 4 kg .. of the first super-blocks, and those of the second 40 lanes on
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_down(a.v[0][i], 40);
      if (kg < 2 && c16 < g.n && c16 < kCols) to(c16, 4 * kg, v);
    } else if (c16 < g.n) {
#pragma unroll
      for (int h = 0; h < RT; ++h) to(c16, h * 16 + 4 * kg, a.v[h]);
    }
  }
};

}  // namespace mmq
