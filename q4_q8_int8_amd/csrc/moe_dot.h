// The vector-ALU form of the experts' products (not part of the ABI): a few columns against RW
// weight rows of one expert, integer dot products on v_dot4_i32_i8.
//
// A matrix instruction costs the same for one column as for sixteen, and the rescale of its
// results too: per 16 rows and 32-block about 20 vector instructions. On the vector ALU a lane
// takes one row and half a super-block: per block 12 instructions to unpack the nibbles and make
// the scales and 12 per column (8 dot products, 4 for the rescale), for 64 (row, block) pairs at a
// time. Up to about 5 columns that is less, and with one token most experts have one column.
//
// Lane l of a wavefront has row l % RW and slice l / RW; a step covers 64 / RW / 2 super-blocks,
// slice q being half q % 2 of super-block q / 2 of the step. Per step a lane loads its row's 64
// nibble bytes and 16-byte header (5 loads of 16 bytes; the lanes of a slice read contiguous
// memory), and the wavefront stages its columns' token bytes [m][slice][128] by direct-to-LDS
// loads and their (da, sa) as float pairs [m][slice][4], which the lanes of a slice read at one
// address. The next step's loads are issued before a step is computed, into a second register set
// and a second LDS buffer. The arithmetic per block is that of mmq_gemv.hip:
//   u = fma(dmv, sa, fma(D, dsv, -1.5*2^23*dsv)),  acc = fma(u, da, acc).
//
// FUSED takes float32 activations and quantizes them itself (the arithmetic of quantize_q8_1,
// quant_device.h): each lane of a slice takes 128 / RW values of the slice's 128, and the lanes of
// a 32-block combine their maximum and integer sum by lane moves.
#pragma once

#include "mmq_device.h"
#include "quant_device.h"

namespace mmq {

constexpr uint32_t kNoRecord = 0xE0000000u;  // past every tile's records: loads give zeros

typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <int RW, int MT, bool FUSED>
struct DotWave {
  static constexpr int kRows = RW;
  static constexpr int kCols = MT;
  static constexpr bool kFused = FUSED;
  static constexpr int SL = 64 / RW;       // slices
  static constexpr int SB = SL / 2;        // super-blocks per step
  static constexpr int kQ = MT * SL * 128;  // LDS: token bytes, then float pairs
  static constexpr int kBuf = kQ + MT * SL * 4 * 8;
  static constexpr int kLds = 2 * kBuf;
  static constexpr int kDma = (MT * SL * 8 + 63) / 64;      // direct-to-LDS loads per step
  static constexpr int kSc = (MT * SL * 4 + 63) / 64;       // (da, sa) pairs per lane
  static constexpr int kXv = FUSED ? 128 / RW / 4 : 1;      // float4 per lane and column
  static_assert(RW == 16 || RW == 8, "rows per wavefront");
  static_assert(!FUSED || MT == 1, "one column from float32");

  // Where the columns come from: a q8 buffer of `rows` x K, or (FUSED) float32 rows of K.
  struct Tokens {
    v4i rq;                        // int8 q, for the direct-to-LDS loads
    __amdgpu_buffer_rsrc_t words;  // packed (da, sa)
    const float4v* x;              // FUSED
    uint32_t K, kb;
  };
  static __device__ __forceinline__ Tokens tokens(const void* p, int rows, int K) {
    Tokens t{};
    t.K = (uint32_t)K;
    t.kb = (uint32_t)(K >> 5);
    if constexpr (FUSED) {
      t.x = static_cast<const float4v*>(p);
    } else {
      const uint8_t* b = static_cast<const uint8_t*>(p);
      t.rq = make_rsrc_sgpr(b, (uint32_t)rows * t.K);
      t.words = make_rsrc(b + (size_t)rows * t.K, (uint32_t)rows * t.kb * 4u);
    }
    return t;
  }

  struct Regs {
    v4i nib[4];
    v4i hdr;
    uint32_t word[kSc];
    float4v xv[kXv];
  };

  struct Acc {
    float v[MT];
  };

  // The columns of a group: n of them (wave-uniform), and the q8 (or x) rows of those that this
  // lane loads for: column (64 i + lane) / (8 SL) of its token bytes, column (64 i + lane) / (4 SL)
  // of its (da, sa) words.
  struct Group {
    uint4v drow, wrow;  // elements 0 .. kDma - 1, 0 .. kSc - 1
    int n, fill0, fill1, fill2;  // (no padding: a copy of padding would go through scratch memory)
  };

  int lane, row, q, hf;
  uint8_t* lds;      // this wavefront's kLds bytes
  uint32_t lds_at;

  __device__ __forceinline__ void init(uint8_t* region, uint32_t at) {
    lane = threadIdx.x & 63;
    row = lane % RW;
    q = lane / RW;
    hf = q & 1;
    lds = region;
    lds_at = at;
  }

  // row_of(m): the row of column m, 0 <= m < n (it may differ by lane).
  template <typename RowOf>
  __device__ __forceinline__ Group group(int n, RowOf row_of) const {
    Group g;
    g.n = n;
    g.fill0 = g.fill1 = g.fill2 = 0;
    g.drow = g.wrow = uint4v{0, 0, 0, 0};
    static_assert(kDma <= 4 && kSc <= 4, "row registers");
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int m = (i * 64 + lane) / (SL * 8);
      g.drow[i] = row_of(m < n ? m : n - 1);
    }
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int m = (i * 64 + lane) / (SL * 4);
      g.wrow[i] = FUSED ? 0u : row_of(m < n ? m : n - 1);
    }
    return g;
  }

  // The parts of a step's loads: step j, rows j0 .. of the tile of `rw`, columns of g. With 16 rows
  // the nibbles are loaded as read once, although an expert of more columns than MT reads them again:
  // the down product of 2 of 8 experts of 4096 x 11008 takes 31.6 us so against 35.2 for 4 tokens, 57.9
  // against 60.7 for 16 (4 columns on average); at 5 columns the two are equal (16 tokens, 4 of 16:
  // 58.2, 58.3), and above this form is not chosen. With 8 rows, whose outputs are small, it made no
  // difference beyond the cache, 31.0 and 30.7 us for 23 tokens, 6 of 64, and cost 5 us of 25 while
  // they fit it.
  static constexpr int kAux = RW == 16 ? kReadOnce : 0;
  struct Src {
    __amdgpu_buffer_rsrc_t rw;
    uint32_t rec;  // the lane's record; past the end of the tile: nothing is loaded
    int j0, j;
  };
  __device__ __forceinline__ Src source(__amdgpu_buffer_rsrc_t rw, int j0, int, int j,
                                        bool any) const {
    return Src{rw, any ? (uint32_t)(j * SB + (q >> 1)) * kRepTileBytes : kNoRecord, j0, j};
  }
  __device__ __forceinline__ void load_nib(const Src& f, int i, Regs& r) const {
    r.nib[i] = buf_load16_aux<kAux>(
        f.rw, f.rec + (2 * hf + (i >> 1)) * 1024 + (i & 1) * 512 + (f.j0 + row) * 16);
  }
  __device__ __forceinline__ void load_hdr(const Src& f, Regs& r) const {
    r.hdr = buf_load16(f.rw, f.rec + kRepNibBytes + (f.j0 + row) * 16);
  }
  __device__ __forceinline__ void load_columns(const Tokens& t, const Group& g, int j, int nsb,
                                               int buf, Regs& r) const {
    if constexpr (FUSED) {
      const int s = j * SB + (q >> 1);
#pragma unroll
      for (int e = 0; e < kXv; ++e) r.xv[e] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
      if (s < nsb) {
        const float4v* p =
            t.x + ((size_t)g.drow[0] * t.K + (size_t)s * 256 + hf * 128) / 4 + row * kXv;
#pragma unroll
        for (int e = 0; e < kXv; ++e) r.xv[e] = p[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kDma; ++i) {
        const int m0 = i * 64 / (SL * 8);
        if (m0 < g.n) {
          const int c = i * 64 + lane, sl = (c / 8) % SL;
          const int sc = j * SB + (sl >> 1);
          if (c < MT * SL * 8)
            dma16(t.rq, lds_at + buf * kBuf + i * 1024,
                  g.drow[i] * t.K + (uint32_t)(sc * 256 + (sl & 1) * 128 + (c & 7) * 16));
        }
      }
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        const int c = i * 64 + lane, m = c / (SL * 4), sl = (c / 4) % SL;
        const int sc = j * SB + (sl >> 1);
        r.word[i] = 0;
        if (m < g.n && sc < nsb)
          r.word[i] = __builtin_bit_cast(
              uint32_t, buf_load_f32(t.words, (g.wrow[i] * t.kb +
                                               (uint32_t)(sc * 8 + (sl & 1) * 4 + (c & 3))) * 4u));
      }
    }
  }
  __device__ __forceinline__ void load_weights(const Src& f, Regs& r) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_nib(f, i, r);
    load_hdr(f, r);
  }

  // What is left of a step's staging once its loads may be waited for.
  __device__ __forceinline__ void finish(const Tokens&, const Group&, const Src&, int buf,
                                         const Regs& r) const {
    uint8_t* b = lds + buf * kBuf;
    asm volatile("" ::: "memory");  // the previous step's LDS reads stay above
    if constexpr (FUSED) {
      float a = 0.0f;
#pragma unroll
      for (int e = 0; e < kXv; ++e) {
        const float4v v = r.xv[e];
        a = fmaxf(a, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
      }
      // the 32 / (4 kXv) lanes of a block: 4 (16 rows) or 2 (8 rows)
      a = fmaxf(a, __int_as_float(dpp<kSwap1>(__float_as_int(a))));
      if constexpr (RW == 16) a = fmaxf(a, __int_as_float(dpp<kSwap2>(__float_as_int(a))));
      const float d = a / 127.0f;                   // IEEE division
      const float id = d > 0.0f ? 1.0f / d : 0.0f;  // IEEE reciprocal (division)
      uint32_t packed[kXv];
      int sum = 0;
#pragma unroll
      for (int e = 0; e < kXv; ++e) {
        const float4v v = r.xv[e];
        const int q0 = quant1(v.x, id), q1 = quant1(v.y, id);
        const int q2 = quant1(v.z, id), q3 = quant1(v.w, id);
        sum += q0 + q1 + q2 + q3;
        packed[e] = (uint32_t)(q0 & 0xFF) | ((uint32_t)(q1 & 0xFF) << 8) |
                    ((uint32_t)(q2 & 0xFF) << 16) | ((uint32_t)(q3 & 0xFF) << 24);
      }
      sum += dpp<kSwap1>(sum);
      if constexpr (RW == 16) sum += dpp<kSwap2>(sum);
      uint32_t* to = reinterpret_cast<uint32_t*>(b + q * 128) + row * kXv;
#pragma unroll
      for (int e = 0; e < kXv; ++e) to[e] = packed[e];
      constexpr int LB = 8 / kXv;  // lanes per block
      if (row % LB == 0)
        reinterpret_cast<float2*>(b + kQ)[q * 4 + row / LB] =
            make_float2((float)(_Float16)d, (float)sum);
    } else {
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        const int c = i * 64 + lane;
        if (c < MT * SL * 4)
          reinterpret_cast<float2*>(b + kQ)[c] =
              make_float2((float)__builtin_bit_cast(_Float16, (uint16_t)(r.word[i] & 0xFFFFu)),
                          (float)((int)r.word[i] >> 16));
      }
    }
    // everything issued has arrived, and the writes are ordered before the step's reads
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // a += step j of group g, whose registers r and LDS buffer `buf` are; each register is loaded for
  // the next step (f, columns gn, into the other buffer; `more`: there is one) once its last use
  // is behind. A lane past the last super-block has zero weights and leaves its sums alone.
  __device__ __forceinline__ void compute(const Group& g, int nsb, int j, int buf, Regs& r, Acc& a,
                                          bool more, const Src& f, const Tokens& t,
                                          const Group& gn) const {
    const bool act = j * SB + (q >> 1) < nsb;
    float(&acc)[MT] = a.v;
    const uint8_t* b = lds + buf * kBuf;
    float dsv[4], dmv[4], nds[4];
    q4k_scales(r.hdr, hf != 0, dsv, dmv);
#pragma unroll
    for (int i = 0; i < 4; ++i) nds[i] = -kBiasF * dsv[i];
    __builtin_amdgcn_sched_barrier(0);
    load_hdr(f, r);
    if (more) load_columns(t, gn, f.j, nsb, buf ^ 1, r);
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      int lo[8], hi[8];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const uint32_t w = (uint32_t)r.nib[2 * gg + (d >> 2)][d & 3];
        lo[d] = (int)(w & 0x0F0F0F0Fu);
        hi[d] = (int)((w >> 4) & 0x0F0F0F0Fu);
      }
      __builtin_amdgcn_sched_barrier(0);  // not before: the registers are in use
      load_nib(f, 2 * gg, r);
      load_nib(f, 2 * gg + 1, r);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m < g.n && act) {
          const v4i* tq = reinterpret_cast<const v4i*>(b + (m * SL + q) * 128 + gg * 64);
          const float4 sc =
              *reinterpret_cast<const float4*>(b + kQ + ((m * SL + q) * 4 + 2 * gg) * 8);
          int S0 = kBiasBits, S1 = kBiasBits;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4i ta = tq[h], tc = tq[2 + h];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              S0 = __builtin_amdgcn_sdot4(lo[4 * h + d], ta[d], S0, false);
              S1 = __builtin_amdgcn_sdot4(hi[4 * h + d], tc[d], S1, false);
            }
          }
          const float t0 = __builtin_fmaf(__int_as_float(S0), dsv[2 * gg], nds[2 * gg]);
          acc[m] = __builtin_fmaf(__builtin_fmaf(dmv[2 * gg], sc.y, t0), sc.x, acc[m]);
          const float t1 = __builtin_fmaf(__int_as_float(S1), dsv[2 * gg + 1], nds[2 * gg + 1]);
          acc[m] = __builtin_fmaf(__builtin_fmaf(dmv[2 * gg + 1], sc.w, t1), sc.z, acc[m]);
        }
      }
    }
  }

  static __device__ __forceinline__ void zero(Acc& a) {
#pragma unroll
    for (int m = 0; m < MT; ++m) a.v[m] = 0.0f;
  }
  // The finished sums, the slices' added pairwise: to(column, row, value), by the row's lane of
  // slice 0.
  template <typename To>
  __device__ __forceinline__ void each(const Group& g, const Acc& a, To to) const {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m < g.n) {
        float v = a.v[m];
        if constexpr (RW == 8) v += __shfl_xor(v, 8);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (q == 0) to(m, row, v);
      }
    }
  }
};

}  // namespace mmq
