// The matrix-unit form of the experts' products (not part of the ABI): up to NT columns against 16
// or 32 weight rows of one expert per wavefront, one v_mfma_i32_16x16x32_i8 per 32-block and 16
// rows. The form of mmq_gemv.hip's decode tile with the columns gathered: 16-byte pieces of any
// row of q8 go to the wavefront's LDS by direct-to-LDS loads. Columns past the expert's are never
// loaded: what LDS holds in their place only reaches result columns that nobody takes.
//
// Per super-block (a step):
//   D   = MFMA_i8(w, q, bias)          S exactly, biased by 1.5*2^23
//   y   = fma(D, da, -1.5*2^23*da)     RN(S * da)
//   acc = fma(y, dsv, acc)
// and two bf16 MFMAs add term2 from the exact three-piece splits of dmv (expanded here from the
// row headers) and of da*sa (in the q8 buffer). Up to 16 columns cost what one does, about 150
// vector instructions per super-block and 16 rows.
//
// Operand layout: A row and B column l % 16 take the 8 k values 8 (l / 16) .. + 7; register r of
// lane l is row 4 (l / 16) + r, column l % 16 of the result.
#pragma once

#include "mmq_device.h"
#include "moe_dot.h"

namespace mmq {

typedef float v4f __attribute__((ext_vector_type(4)));

// KS = 2: 8 weight rows and two super-blocks at a time. Operand rows 0..7 are the rows of the first
// super-block and 8..15 the same rows of the second, operand columns 0..7 the columns of the first
// and 8..15 of the second; the two diagonal 8 x 8 quarters of the result are the two super-blocks'
// sums, the others are left. An expert of up to 8 columns costs as much per weight as with 16 rows,
// and an output of few rows gives twice the workgroups.
// NT counts the staged columns (KS of them per column of the product); NBUF: LDS buffers for them.
template <int RT, int NT, int KS = 1, int NBUF = 2>
struct MfmaWave {
  static_assert(KS == 1 || (KS == 2 && RT == 1), "forms");
  static constexpr int kRows = 16 * RT / KS;
  static constexpr int kCols = NT / KS;
  static constexpr bool kFused = false;
  static constexpr int SB = KS;
  // LDS: per 16 rows the expanded scales (dsv f32 [8][16], the dmv pieces bf16 [3][16][8]), then
  // twice the columns' operands of a super-block: int8 [NT][256], the 16-byte chunk c of column t
  // at chunk c ^ t, and the da*sa pieces bf16 [3][NT][8]
  static constexpr int kDsv = 8 * 16 * 4;
  static constexpr int kScale = kDsv + 3 * 16 * 8 * 2;
  static constexpr int kBuf = NT * 256 + 3 * NT * 16;
  static constexpr int kLds = RT * kScale + NBUF * kBuf;

  struct Tokens {
    v4i rq, rpc;                    // q and the da*sa pieces, for the direct-to-LDS loads
    __amdgpu_buffer_rsrc_t rwd;     // packed (da, sa) words
    uint32_t rows, K, kb;
  };
  static __device__ __forceinline__ Tokens tokens(const void* p, int rows, int K) {
    const uint8_t* base = static_cast<const uint8_t*>(p);
    Tokens q;
    q.rows = (uint32_t)rows;
    q.K = (uint32_t)K;
    q.kb = (uint32_t)(K >> 5);
    q.rq = make_rsrc_sgpr(base, q.rows * q.K);
    q.rpc = make_rsrc_sgpr(base + q8_pieces_offset(rows, K), q.rows * (q.K >> 8) * 48u);
    q.rwd = make_rsrc(base + (size_t)rows * K, q.rows * q.kb * 4u);
    return q;
  }

  // n columns (wave-uniform). Staged column t is column t % kCols of super-block t / kCols of the
  // step. Lane l stages 16-byte chunks of staged columns 4 i + l / 16 and, below 3 NT, piece l / NT
  // of staged column l % NT; as an operand lane it has staged column `col`.
  struct Group {
    uint4v drow;               // q8 row of staged column 4 i + l / 16
    uint32_t prow, row;        // q8 row of staged column l % NT, of `col`
    int n, fill;               // (no padding: a copy of padding would go through scratch memory)
  };
  template <typename RowOf>
  __device__ __forceinline__ Group group(int n, RowOf row_of) const {
    Group g;
    g.n = n;
    g.fill = 0;
    auto at = [&](int t) { return row_of(t % kCols < n ? t % kCols : n - 1); };
    g.drow = uint4v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NT / 4; ++i) g.drow[i] = at(4 * i + (lane >> 4));
    g.prow = at(lane % NT);
    g.row = at(col);
    return g;
  }

  struct Regs {
    uint2 nib[RT][4];
    v4i hdr[RT];
    v4i wd[2];
  };
  struct Acc {
    v4f v[RT];
  };

  int lane, c16, kg;
  int row, sel, col;  // operand row's weight row, its super-block of the step, the staged column
  uint8_t* lds;
  uint32_t lds_at;
  v4i bias;

  __device__ __forceinline__ void init(uint8_t* region, uint32_t at) {
    lane = threadIdx.x & 63;
    c16 = lane & 15;
    kg = lane >> 4;
    row = KS == 2 ? c16 & 7 : c16;
    sel = KS == 2 ? c16 >> 3 : 0;
    col = KS == 2 ? sel * kCols + (c16 & (kCols - 1)) : c16 & (NT - 1);
    lds = region;
    lds_at = at;
    bias = v4i{kBiasBits, kBiasBits, kBiasBits, kBiasBits};
    asm volatile("" : "+v"(bias));
  }

  // The parts of a step's loads: super-block s, rows j0 .. of the tile of `rw`, columns of g.
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
  __device__ __forceinline__ void load_nib(const Src& f, int i, Regs& r) const {
#pragma unroll
    for (int h = 0; h < RT; ++h)
      r.nib[h][i] = __builtin_bit_cast(
          uint2, buf_load_f32x2(f.rw, f.rec + i * 1024 + (kg >> 1) * 512 +
                                          (f.j0 + h * 16 + row) * 16 + (kg & 1) * 8));
  }
  __device__ __forceinline__ void load_hdr(const Src& f, Regs& r) const {
#pragma unroll
    for (int h = 0; h < RT; ++h)
      r.hdr[h] = buf_load16(f.rw, f.rec + kRepNibBytes + (f.j0 + h * 16 + row) * 16);
  }
  __device__ __forceinline__ void load_words(const Tokens& t, const Group& g, int s, bool ok, int i,
                                             Regs& r) const {
    const uint32_t at = (g.row * t.kb + (uint32_t)(s + sel) * 8u) * 4u + 16u * i;
    r.wd[i] = buf_load16(t.rwd, ok ? at : kNoRecord);  // no super-block: scales of 0
  }
  __device__ __forceinline__ void stage_columns(const Tokens& t, const Group& g, int s,
                                                int buf) const {
    const uint32_t tok = lds_at + RT * kScale + (NBUF == 2 ? buf * kBuf : 0);
#pragma unroll
    for (int i = 0; i < NT / 4; ++i) {
      if (4 * i % kCols < g.n) {  // wave-uniform
        const int c = 4 * i + (lane >> 4), ch = (lane & 15) ^ c;
        dma16(t.rq, tok + i * 1024,
              g.drow[i] * t.K + (uint32_t)(s + c / kCols) * 256u + (uint32_t)ch * 16u);
      }
    }
    if (lane < 3 * NT)
      dma16(t.rpc, tok + NT * 256,
            (((uint32_t)(s + lane % NT / kCols) * 3u + (uint32_t)(lane / NT)) * t.rows + g.prow) *
                16u);
  }
  __device__ __forceinline__ void load_weights(const Src& f, Regs& r) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_nib(f, i, r);
    load_hdr(f, r);
  }
  // What of step j's columns is loaded ahead of finish().
  __device__ __forceinline__ void load_columns(const Tokens& t, const Group& g, int j, int nsb,
                                               int buf, Regs& r) const {
    const bool ok = KS == 1 || KS * j + sel < nsb;
    load_words(t, g, KS * j, ok, 0, r);
    load_words(t, g, KS * j, ok, 1, r);
    if (NBUF == 2) stage_columns(t, g, KS * j, buf);
  }

  // Once the previous step is computed: wait for the loads and expand the scales, lane (c16, kg)
  // sub-blocks 2 kg and 2 kg + 1 of row c16 of each half.
  __device__ __forceinline__ void finish(const Tokens& t, const Group& g, const Src& f, int,
                                         const Regs& r) const {
    asm volatile("" ::: "memory");  // the previous step's LDS reads stay above
    if (NBUF == 1) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): ... and are done before the buffer's loads
      stage_columns(t, g, f.s, 0);
      asm volatile("" ::: "memory");
    }
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      const uint32_t w0 = (uint32_t)r.hdr[h][0], s0 = (uint32_t)r.hdr[h][1],
                     s1 = (uint32_t)r.hdr[h][2], s2 = (uint32_t)r.hdr[h][3];
      const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)(w0 & 0xFFFFu));
      const float dm = -(float)__builtin_bit_cast(_Float16, (uint16_t)(w0 >> 16));
      // the packed scales as q4k_scales reads them, then this lane's two of each four
      const uint32_t hm = 0u - (uint32_t)(kg >= 2), sh = 16u * (uint32_t)(kg & 1);
      const uint32_t sc = ((((s2 & 0x0F0F0F0Fu) | ((s0 >> 2) & 0x30303030u)) & hm) |
                           ((s0 & 0x3F3F3F3Fu) & ~hm)) >> sh;
      const uint32_t mm = (((((s2 >> 4) & 0x0F0F0F0Fu) | ((s1 >> 2) & 0x30303030u)) & hm) |
                           ((s1 & 0x3F3F3F3Fu) & ~hm)) >> sh;
      float* sd = reinterpret_cast<float*>(lds + h * kScale);
      sd[(2 * kg) * 16 + c16] = d * (float)(sc & 0xFFu);
      sd[(2 * kg + 1) * 16 + c16] = d * (float)((sc >> 8) & 0xFFu);
      uint32_t pa[3], pb[3];
      bf16_trunc3(dm * (float)(mm & 0xFFu), pa[0], pa[1], pa[2]);
      bf16_trunc3(dm * (float)((mm >> 8) & 0xFFu), pb[0], pb[1], pb[2]);
      uint32_t* sp = reinterpret_cast<uint32_t*>(lds + h * kScale + kDsv);
#pragma unroll
      for (int i = 0; i < 3; ++i) sp[(i * 16 + c16) * 4 + kg] = pack_hi16(pa[i], pb[i]);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the writes are done
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // acc += the step whose registers r, LDS buffer `buf` are; each register is loaded for the next
  // step (f, columns gn, into the other buffer; `more`: there is one) once its last use is behind.
  __device__ __forceinline__ void compute(const Group&, int, int, int buf, Regs& r, Acc& acc,
                                          bool more, const Src& f, const Tokens& t,
                                          const Group& gn) const {
    if (NBUF == 2 && more) stage_columns(t, gn, f.s, buf ^ 1);
    load_hdr(f, r);
    const uint8_t* stok = lds + RT * kScale + (NBUF == 2 ? buf * kBuf : 0);
    // term2 piece pairs of this lane's k-group: (0,0) (0,1) (1,0) (0,2) in the first instruction,
    // (1,1) (2,0) and two zero groups in the second
    const int ia1 = kg == 2 ? 1 : 0, jb1 = kg == 1 ? 1 : (kg == 3 ? 2 : 0);
    const int ia2 = kg == 1 ? 2 : 1, jb2 = kg == 0 ? 1 : 0;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint2 tb = *reinterpret_cast<const uint2*>(
          stok + col * 256 + (((2 * b + (kg >> 1)) ^ col) << 4) + (kg & 1) * 8);
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
        const v4f dsv = *reinterpret_cast<const v4f*>(lds + h * kScale + (b * 16 + 4 * kg) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = __builtin_fmaf(__int_as_float(D[i]), da, nda);
          acc.v[h][i] = __builtin_fmaf(y, dsv[i], acc.v[h][i]);
        }
      }
      if (b & 1) {
        __builtin_amdgcn_sched_barrier(0);  // not before: the registers are in use
        load_nib(f, b >> 1, r);
        if ((b & 3) == 3) load_words(t, gn, f.s, f.ok, b >> 2, r);
      }
    }
    const uint8_t* pc = stok + NT * 256;
    const v4i pb0 = *reinterpret_cast<const v4i*>(pc + (jb1 * NT + col) * 16);
    const v4i pb1 = *reinterpret_cast<const v4i*>(pc + (jb2 * NT + col) * 16);
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      const uint8_t* sp = lds + h * kScale + kDsv;
      const v4i pa0 = *reinterpret_cast<const v4i*>(sp + (ia1 * 16 + c16) * 16);
      v4i pa1 = *reinterpret_cast<const v4i*>(sp + (ia2 * 16 + c16) * 16);
      if (kg >= 2) pa1 = v4i{0, 0, 0, 0};
      acc.v[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(v8bf, pa0), __builtin_bit_cast(v8bf, pb0), acc.v[h], 0, 0, 0);
      acc.v[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(v8bf, pa1), __builtin_bit_cast(v8bf, pb1), acc.v[h], 0, 0, 0);
    }
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
