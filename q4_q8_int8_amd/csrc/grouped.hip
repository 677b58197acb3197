// The q4_K x q8_1 product grouped by expert: out[p] = act(x[src(p)] W(e)^T), or its gated form, for
// every pair p of the groups with an expert e, the rows of one expert being one ragged matrix.
//
// The arithmetic is the tile of mmq_gemm.hip, per element the same operations in the same order (its
// comment has the mathematics: one int8 MFMA per 32-block, two FMAs per element to rescale it, term2
// on the bf16 unit, three instructions per super-block). What differs is which rows a workgroup has and how
// they get into LDS:
//
// - The host knows the pairs, not how they fall on the experts. The grid covers the most tiles that
//   they can form (P / BM + min(E, P) for tiles of BM rows); a workgroup finds its expert and rows
//   from the offsets of the groups, one work-item per expert and one prefix sum, and ends at once
//   where there is no such tile.
// - An expert's rows are cut into tiles of 32 TT rows, the last one of the 32-row parts it needs: the
//   tile's code exists for 1 .. TT parts and a workgroup branches to its own, so a tile of few rows
//   does not pay for the rescale of many. In the forms of 32 rows a tile of at most 16 uses 16 x 16
//   instructions, half the elements to rescale (experts of 12 rows each, 22016 x 4096, 8 of them: 114 ->
//   106 us; 2048 x 2048, 64 of them: 44.9 -> 43.9; no difference above 16).
// - The rows are gathered by the loads into LDS: each lane's address has its row's place in the q8
//   buffer, taken from the groups once per workgroup. quantize_q8_1's (da, nda) plane is block-major
//   for contiguous rows; here it is row-major, 16 bytes holding two blocks of a row, staged as
//   [4 pairs of blocks][BM] of 16 bytes and read as one (read as two halves of 8 bytes, they met two ways in
//   the LDS banks: 2048 tokens, 2 of 8, 1090 and 633 us against 1069 and 621). Tokens are quantized once,
//   not once per slot.
// - Workgroups go to the XCDs in turn. Each XCD gets a contiguous range of the tiles in the order
//   (block of weight-tile groups, expert, group, rows), so the row tiles that share weights run on one L2.
//
// With few rows per expert it is bound by the weights' bytes: 64 experts, 100 tokens of 8 slots, D = 2048,
// F = 1024 move their 151 MB of gate and up weights in 40 to 51 us with the quantization (3.0 to 3.8 TB/s, a
// large copy moving 5.2; VALU 65 % busy). With many it is bound as the plain product is, by the rescale's
// vector instructions: 2048 tokens, 2 of 8, 4096 -> 2 x 11008, 1056 us, 350 GMAC/ms, VALU 93 % busy (the
// plain product reaches 377). Its clock is then 1.45 to 1.6 GHz by the power that the card allows, against
// 2.0 to 2.1 in a single launch, which neither a longer pipeline (a workgroup that walks several tiles, with
// the next one's first stage under the last super-block: 138 -> 139 us on 64 experts of 64 rows) nor other
// tiles (64 rows, 4 or 8 wavefronts, 12 wavefronts on three SIMD slots: within 3 %) get past.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "epilogue.h"
#include "grouped_internal.h"
#include "mmq_device.h"

namespace mmq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void set_priority(int p) {
  if (p >= 3) __builtin_amdgcn_s_setprio(3);
  else if (p == 2) __builtin_amdgcn_s_setprio(2);
  else if (p == 1) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

// The shape of a workgroup: CW wavefronts side by side, one 32-row weight tile each, for every of KS
// ranges of K, and TMAX 32-row parts of an expert's rows at most; WAVES wavefronts to a SIMD.
template <int TMAX_, int CW_, int KS_, int WAVES_>
struct Form {
  static constexpr int TMAX = TMAX_, CW = CW_, KS = KS_, NW = CW_ * KS_, WAVES = WAVES_;
  static constexpr int BM = 32 * TMAX;
  static constexpr bool kLean = WAVES >= 4;  // 128 registers to a wavefront
  // Weight-tile groups that an expert's tiles are gone through with before the next expert's: with 8 the
  // narrow form takes 2 to 4 % less (777 tokens, 6 of 64, 1280 -> 2048: 84.0 -> 80.8 us) from its rows
  // being in the L2; with 1 the wide form's short tiles, the last ones of the experts, are spread evenly
  // over the XCDs (2048 tokens, 2 of 8: 11008 -> 4096 626 against 677 us with 8, 4096 -> 22016 1097
  // against 1086).
  static constexpr int kBlock = kLean ? 8 : 1;
  // Whether the last round of an XCD's tiles is cut finer (find_tile).
  static constexpr bool kTail = TMAX == 4;
  // One stage: per range of K the int8 token tile [BM][272], the (da, nb) pairs [4][BM][2 blocks][2]
  // and the token pieces [3][BM][8]; then the wavefronts' 32 row headers. Behind the two stages the
  // expanded weight scales, which only their wavefront uses, one super-block at a time; then the
  // tile's rows, each its pair and its row of the q8 buffer.
  static constexpr int kTokA = BM * kRowStride, kTokDa = BM * 64, kTokP = BM * 48;
  static constexpr int kTokens = kTokA + kTokDa + kTokP;
  static constexpr int kStage = KS * kTokens + NW * kRepHdrBytes;
  static constexpr int kExpanded = kWDsvBytes + kWPieceBytes;
  static constexpr int kRowsAt = 2 * kStage + NW * kExpanded;
  static constexpr int kLds = kRowsAt + BM * (int)sizeof(int2);
  static constexpr int kADma = (BM * (kRowStride / 16) + 63) / 64;  // wavefront-wide instructions
  static constexpr int kDaDma = (4 * BM + 63) / 64, kPDma = (3 * BM + 63) / 64;
  static constexpr int kAOps = (kADma + CW - 1) / CW, kDaOps = (kDaDma + CW - 1) / CW;
  static constexpr int kPOps = (kPDma + CW - 1) / CW;
  // what a stage loads into LDS, as single instructions of a wavefront: its row headers and its share
  // of the tokens
  static constexpr int kOps = 1 + kAOps + kDaOps + kPOps;
};

struct Args {
  const int8_t* qs;
  const float* da;
  const uint16_t* pieces;
  const int* groups;
  const uint8_t* w;
  float* out;
  int P, E, N, K, q_rows, per_row, gn, order_at;
  int most;  // the most tiles of a weight-tile group that the pairs can form
  int slots;  // workgroups that an XCD runs at a time (F::kTail)
};

// A tile: its expert, its first row in the order, its rows (0: none) and its weight-tile group.
struct Pick {
  int expert, first, rows, tn;
};

// The tile of this workgroup: each wavefront looks at 64 experts at a time, one to a lane. The offsets
// are only used inside [0, P], so that groups of nonsense select nonsense rows of this product and no
// others. In LDS before the first stage is loaded.
struct SearchLds {
  int totals[kGroupMaxExperts / 64];
  Pick pick;
};
template <class F>
__device__ __forceinline__ Pick find_tile(SearchLds& sh, const Args& g) {
  constexpr int NCH = kGroupMaxExperts / 64, CH = (NCH + F::NW - 1) / F::NW;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int lo[CH], n[CH], incl[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (wave + c * F::NW) * 64 + lane;
    lo[c] = n[c] = 0;
    if (e < g.E) {
      lo[c] = min(max(g.groups[e], 0), g.P);
      n[c] = min(max(g.groups[e + 1], lo[c]), g.P) - lo[c];
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    incl[c] = (n[c] + F::BM - 1) / F::BM;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(incl[c], d);
      if (lane >= d) incl[c] += o;
    }
    if (lane == 63 && wave + c * F::NW < NCH) sh.totals[wave + c * F::NW] = incl[c];
  }
  if (threadIdx.x == 0) sh.pick.rows = 0;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < NCH; ++w) {
    const int v = sh.totals[w];
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (w < wave + c * F::NW) incl[c] += v;
    all += v;
  }
  all = min(all, g.most);  // what the grid covers (offsets of nonsense may ask for more)
  // tiles in the order (weight-tile group's block, expert, group, rows), one contiguous range per XCD
  const unsigned total = (unsigned)all * (unsigned)g.gn;
  const unsigned per_xcd = (total + 7u) >> 3;
  unsigned k = blockIdx.x >> 3;
  // The tiles of an XCD's last round, where they fill a half or a quarter of it, as 2 or 4 workgroups of 64 or
  // 32 rows each (1500 tokens, 2 of 8: 4096 -> 2 x 4096 345 -> 322 us, 4096 -> 4096 213.5 and 214.8; 2048 tokens,
  // 4096 -> 2 x 11008 1106 -> 1099, 11008 -> 4096 630 -> 626 and, of other counts, 636 -> 543). Fuller rounds
  // stay whole: finer workgroups unpack a tile's weights and expand its scales again, each for itself.
  int part = 0, shift = 0;
  if constexpr (F::kTail) {
    const unsigned last = per_xcd % (unsigned)g.slots, whole = per_xcd - last;
    shift = 4 * last <= (unsigned)g.slots ? 2 : 2 * last <= (unsigned)g.slots ? 1 : 0;
    if (k >= whole) {
      part = (int)((k - whole) & ((1u << shift) - 1u));
      k = whole + ((k - whole) >> shift);
    } else {
      shift = 0;
    }
  }
  const unsigned idx = (blockIdx.x & 7u) * per_xcd + k;
  if (k < per_xcd && idx < total) {
    const int block = (int)(idx / (unsigned)(all * F::kBlock));
    const int at = (int)(idx - (unsigned)block * (unsigned)(all * F::kBlock));
    const int wide = min(F::kBlock, g.gn - block * F::kBlock);  // groups of this block
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int mine = (n[c] + F::BM - 1) / F::BM;
      const int local = at - (incl[c] - mine) * wide;
      if (local >= 0 && local < mine * wide) {
        const int tn = local / mine, u = local - tn * mine;
        const int row = u * F::BM + part * (F::BM >> shift);
        sh.pick = Pick{(wave + c * F::NW) * 64 + lane, lo[c] + row,
                       min(n[c] - row, F::BM >> shift), block * F::kBlock + tn};
      }
    }
  }
  __syncthreads();
  const Pick p = sh.pick;
  return Pick{__builtin_amdgcn_readfirstlane(p.expert), __builtin_amdgcn_readfirstlane(p.first),
              __builtin_amdgcn_readfirstlane(p.rows), __builtin_amdgcn_readfirstlane(p.tn)};
}

// The rows of a tile, each its pair and its row of the q8 buffer; -1 and the buffer's end past the last.
template <class F>
__device__ __forceinline__ int2 load_row(const Args& g, const Pick& t) {
  const int i = threadIdx.x;
  int p = -1;
  if (i < t.rows) p = g.groups[g.order_at + t.first + i];
  if (p < 0 || p >= g.P) return make_int2(-1, g.q_rows);
  return make_int2(p, (int)((unsigned)p / (unsigned)g.per_row));
}

// What a wavefront loads for a tile.
template <class F>
struct Loads {
  v4i rq, rda, rtp, rwd;
  __amdgpu_buffer_rsrc_t rw;
  uint32_t a_off[F::kAOps], da_off[F::kDaOps], tp_off[F::kPOps];
  uint32_t tp_step;
  int parts, slots, cw, wave, lane;
  bool works;  // whether the wavefront has a weight tile
  uint32_t lds0, tok_at, hdr_at;

  __device__ __forceinline__ void init(const uint8_t* smem, const Args& g) {
    const uint32_t M = (uint32_t)g.q_rows, K = (uint32_t)g.K;
    rq = make_rsrc_sgpr(g.qs, M * K);
    rda = make_rsrc_sgpr(g.da, M * K >> 2);
    rtp = make_rsrc_sgpr(g.pieces, M * (K >> 8) * 48u);
    tp_step = M * 48u;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    cw = F::KS == 1 ? wave : wave % F::CW;
    lds0 = lds_addr(smem);
    tok_at = (uint32_t)((F::KS == 1 ? 0 : wave / F::CW) * F::kTokens);
    hdr_at = (uint32_t)(F::KS * F::kTokens + wave * kRepHdrBytes);
  }
  // The tile's weights.
  __device__ __forceinline__ void aim(const Args& g, const Pick& t) {
    const int ntiles = (g.N + 31) >> 5;
    works = t.tn * F::CW + cw < ntiles;  // one without loads tokens for the others
    const int wt = works ? t.tn * F::CW + cw : ntiles - 1;
    const size_t tile_bytes = (size_t)(g.K >> 8) * kRepTileBytes;
    const uint8_t* wtile = g.w + ((size_t)t.expert * ntiles + wt) * tile_bytes;
    rwd = make_rsrc_sgpr(wtile, (uint32_t)tile_bytes);
    rw = make_rsrc(wtile, (uint32_t)tile_bytes);
    parts = (t.rows + 31) >> 5;
    slots = (t.rows <= 16 ? 16 : parts * 32) * 17;
  }
  // Its tokens: a row past the last, and the padding, read past the buffers' ends (zero), and stay there
  // with every super-block.
  __device__ __forceinline__ void aim(const Args& g, const int2* rows) {
    const uint32_t M = (uint32_t)g.q_rows, K = (uint32_t)g.K;
#pragma unroll
    for (int j = 0; j < F::kAOps; ++j) {  // slot q holds chunk q % 17 of row q / 17
      const int q = (cw + j * F::CW) * 64 + lane;
      const int row = q / 17, c = q - row * 17;
      const uint32_t src = row < F::BM ? (uint32_t)rows[row].y : M;
      a_off[j] = c < 16 && src < M ? src * K + c * 16 : M * K;
    }
#pragma unroll
    for (int j = 0; j < F::kDaOps; ++j) {  // pair of blocks q / BM of row q % BM
      const int q = (cw + j * F::CW) * 64 + lane;
      const uint32_t src = q < 4 * F::BM ? (uint32_t)rows[q % F::BM].y : M;
      da_off[j] = src < M ? src * (K >> 2) + (q / F::BM) * 16 : M * K >> 2;
    }
#pragma unroll
    for (int j = 0; j < F::kPOps; ++j) {  // piece q / BM of row q % BM
      const int q = (cw + j * F::CW) * 64 + lane;
      const uint32_t src = q < 3 * F::BM ? (uint32_t)rows[q % F::BM].y : M;
      tp_off[j] = src < M ? ((uint32_t)(q / F::BM) * M + src) * 16u : M * (K >> 8) * 48u;
    }
  }
  // Instruction v of super-block s into stage p; those of rows that the tile does not have are left out.
  __device__ __forceinline__ void issue(int v, int s, int p) const {
    const uint32_t st = lds0 + (uint32_t)p * F::kStage + tok_at;
    if (v < 1) {
      if (lane < 32)
        dma16(rwd, lds0 + (uint32_t)p * F::kStage + hdr_at,
              (uint32_t)s * kRepTileBytes + kRepNibBytes + lane * 16);
      return;
    }
    v -= 1;
    if (v < F::kAOps) {
      const int k = cw + v * F::CW;
      if (k * 64 < slots) dma(rq, st, k, F::BM * 17, a_off[v] + (uint32_t)s * 256);
      return;
    }
    v -= F::kAOps;
    if (v < F::kDaOps) {
      const int k = cw + v * F::CW;
      if (k < F::kDaDma) dma(rda, st + F::kTokA, k, 4 * F::BM, da_off[v] + (uint32_t)s * 64);
      return;
    }
    v -= F::kDaOps;
    const int k = cw + v * F::CW;
    if (k < F::kPDma)
      dma(rtp, st + F::kTokA + F::kTokDa, k, 3 * F::BM, tp_off[v] + (uint32_t)s * tp_step);
  }
  // slots 64 k .. 64 k + 63, of which `slots` exist
  __device__ __forceinline__ void dma(v4i r, uint32_t lds, int k, int slots, uint32_t off) const {
    if (k * 64 + lane < slots) dma16(r, lds + k * 1024, off);
  }
  __device__ __forceinline__ v4i nibbles(int s, int gi) const {
    return buf_load16(rw, (uint32_t)s * kRepTileBytes + gi * 1024 + lane * 16);
  }
  // The same two blocks for the tile of 16 rows: the lane (r, c) has values 8 c .. 8 c + 7 of both of weight
  // row r in x, y, and of row 16 + r in z, w.
  __device__ __forceinline__ v4i nibbles16(int s, int gi) const {
    const int at = gi * 1024 + (lane >> 5) * 512 + (lane & 15) * 16 + ((lane >> 4) & 1) * 8;
    const int so = s * kRepTileBytes;
    const uint2 a =
        __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rw, at, so, 0));
    const uint2 b =
        __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rw, at + 256, so, 0));
    return v4i{(int)a.x, (int)a.y, (int)b.x, (int)b.y};
  }
};

// The sums of a tile of TT parts over super-blocks s0 .. s1 - 1, the first of which is in stage 0 and, its
// nibbles, in raw; `steps` barriers.
template <class F, int TT>
__device__ __forceinline__ void sums(uint8_t* smem, const Loads<F>& ld, int s0, int s1, int steps,
                                     v4i (&raw)[4], v16f (&acc)[TT]) {
  constexpr int NS = 8 * TT;  // (block, token tile) steps per super-block
  constexpr bool LEAN = F::kLean;
  const int lane = ld.lane, h = lane >> 5, l32 = lane & 31;
  // The next stage's instructions are spread over a super-block's steps, three at a time, as in
  // mmq_gemm.hip.
  auto op_step = [](int v) { return ((v / 3) * 2 * TT < NS - 1) ? (v / 3) * 2 * TT : NS - 1; };
  v16i bias;
#pragma unroll
  for (int r = 0; r < 16; ++r) bias[r] = kBiasBits;
  asm volatile("" : "+v"(bias));  // stays in vector registers, as in mmq_gemm.hip
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.0f;

  // The nibbles of the next stage: in place as they are used up (the last through nib3), or, where a
  // super-block is too short for that (one token tile), all at the first step through a second set.
  constexpr bool ENIB = TT == 1;
  v4i nib3 = raw[3], rawB[ENIB ? 4 : 1];
  for (int i = 0; i < steps; ++i) {
    const int s = s0 + i, p = i & 1;
    if constexpr (!ENIB) raw[3] = nib3;
    const bool more = s + 1 < s1;
    if ((F::KS == 1 || s < s1) && ld.works) {
      const uint8_t* st = smem + p * F::kStage + ld.tok_at;
      const uint8_t* sArow = st + l32 * kRowStride + h * 16;
      const uint8_t* sDa = st + F::kTokA;
      const uint8_t* sTp = st + F::kTokA + F::kTokDa;
      uint8_t* sW = smem + 2 * F::kStage + ld.wave * F::kExpanded;
      const float* sWw = reinterpret_cast<const float*>(sW);
      // (the wavefront's reads of the last super-block's scales came before the barrier)
      auto expand_scales = [&]() {
        const v4i hdr =
            *reinterpret_cast<const v4i*>(smem + p * F::kStage + ld.hdr_at + l32 * 16);
        q4k_stage_scales(hdr, l32, h != 0, sW);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      };
      auto wop_of = [&](int b) -> v4i {
        const v4i rr = raw[b >> 1];
        return (b & 1) ? ((rr >> 4) & 0x0F0F0F0F) : (rr & 0x0F0F0F0F);
      };
      auto top_of = [&](int n) -> v4i {
        const int b = n / TT, t = n % TT;
        return *reinterpret_cast<const v4i*>(sArow + t * 32 * kRowStride + b * 32);
      };
      float2 odd[TT];  // of the second block, read with the first's
      auto da_of = [&](int n) -> float2 {
        const int b = n / TT, t = n % TT;
        if (b & 1) return odd[t];
        const float4 v = *reinterpret_cast<const float4*>(sDa + ((b >> 1) * F::BM + t * 32 + l32) * 16);
        odd[t] = make_float2(v.z, v.w);
        return make_float2(v.x, v.y);
      };
      auto dsv_of = [&](int b, float (&d)[16]) {
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          const float4 a = *reinterpret_cast<const float4*>(sWw + b * 32 + 8 * gi + 4 * h);
          d[4 * gi + 0] = a.x; d[4 * gi + 1] = a.y; d[4 * gi + 2] = a.z; d[4 * gi + 3] = a.w;
        }
      };

      // Entering step n = b*TT + t: D(n) has been issued, the token operand of step n+1 and da of
      // step n are in registers; dsv[b & 1] holds block b's weight scales. LEAN, four wavefronts to a
      // SIMD: the others cover a step's latency instead.
      v16i Dn;
      v4i tnext;
      float2 da;
      float dsv[LEAN ? 1 : 2][16];
      if constexpr (!LEAN) {
        Dn = __builtin_amdgcn_mfma_i32_32x32x32_i8(wop_of(0), top_of(0), bias, 0, 0, 0);
        asm volatile("" : "+v"(Dn));  // issued here, not sunk below the expansion
        tnext = top_of(1 % NS);
        da = da_of(0);
      }
      expand_scales();
      dsv_of(0, dsv[0]);
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int b = n / TT, t = n % TT;
        if (n % 2 == 0) set_priority(3 - (n % 8) / 2);  // the pair of a SIMD keeps step
        if (more) {
          if constexpr (ENIB) {
            if (n == 0) {
#pragma unroll
              for (int gi = 0; gi < 4; ++gi) rawB[gi] = ld.nibbles(s + 1, gi);
            }
          }
#pragma unroll
          for (int v = 0; v < F::kOps; ++v)
            if (op_step(v) == n) ld.issue(v, s + 1, p ^ 1);
          if constexpr (!ENIB) {
            if (op_step(F::kOps) == n) nib3 = ld.nibbles(s + 1, 3);
#pragma unroll
            for (int gi = 0; gi < 3; ++gi)
              if (n == (2 * gi + 2) * TT) raw[gi] = ld.nibbles(s + 1, gi);
          }
        }
        v16i D;
        float2 dac;  // (da, nb)
        if constexpr (LEAN) {
          v4i top = top_of(n);
          asm volatile("" : "+v"(top));  // the steps stay in order
          D = __builtin_amdgcn_mfma_i32_32x32x32_i8(wop_of(b), top, bias, 0, 0, 0);
          dac = da_of(n);
          if (t == 0 && b > 0) dsv_of(b, dsv[0]);
        } else {
          D = Dn;
          dac = da;
          if (n + 1 < NS) {
            Dn = __builtin_amdgcn_mfma_i32_32x32x32_i8(wop_of((n + 1) / TT), tnext, bias, 0, 0, 0);
            da = da_of(n + 1);
          }
          if (n + 2 < NS) tnext = top_of(n + 2);
          if (t == 0 && b + 1 < 8) dsv_of(b + 1, dsv[(b + 1) & 1]);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float y = __builtin_fmaf(__int_as_float(D[r]), dac.x, dac.y);
          acc[t][r] = __builtin_fmaf(y, dsv[LEAN ? 0 : b & 1][r], acc[t][r]);
        }
        if (b == 1 || b == 3 || b == 5) {  // a third of term2, the piece pairs of mmq_gemm.hip
          const int u = b >> 1;
          const int ia = u == 0 ? 0 : (u == 1 ? 1 - h : 1 + h);
          const int jb = u == 0 ? h : (u == 1 ? 2 * h : 1 - h);
          const v8bf wa = *reinterpret_cast<const v8bf*>(sW + kWDsvBytes + (ia * 32 + l32) * 16);
          const v8bf tb =
              *reinterpret_cast<const v8bf*>(sTp + (jb * F::BM + t * 32 + l32) * 16);
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa, tb, acc[t], 0, 0, 0);
        }
      }
    } else if (more) {
#pragma unroll
      for (int v = 0; v < F::kOps; ++v) ld.issue(v, s + 1, p ^ 1);
    }

    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_s_waitcnt(0);  // this wavefront's loads of the next stage have landed
    __syncthreads();                // ... and everyone's; this stage is no longer read
    if constexpr (ENIB) {
#pragma unroll
      for (int gi = 0; gi < 4; ++gi) raw[gi] = rawB[gi];
    }
  }
}

// The same for a tile of at most 16 rows: the 32 weight rows are two tiles of 16 x 16, half the elements to
// rescale. Lane (r, c) has token r and, in acc[w], weight rows 16 w + 4 c .. + 3. raw as nibbles16. Every
// element's operations are those of sums, in their order, so that a row's bits do not go by how many other
// rows its tile has: term2 in the same three steps of 16 products, whose sum the 16 x 16 x 16 and the 32 x 32 x
// 16 instruction round alike (the same bits in 25 million sums of exponents up to 2^+-60). 32 products at a time
// round otherwise.
template <class F>
__device__ __forceinline__ void sums16(uint8_t* smem, const Loads<F>& ld, int s0, int s1, int steps,
                                       v4i (&raw)[4], v4f (&acc)[2]) {
  const int lane = ld.lane, r16 = lane & 15, c = lane >> 4;
  v4i bias;
#pragma unroll
  for (int r = 0; r < 4; ++r) bias[r] = kBiasBits;
  asm volatile("" : "+v"(bias));
  acc[0] = acc[1] = v4f{0.f, 0.f, 0.f, 0.f};
  // which half of a third's 16 products, two piece pairs of 8 blocks each, the lane holds four of
  const int h = c >> 1, part = (c & 1) * 8;
  for (int i = 0; i < steps; ++i) {
    const int s = s0 + i, p = i & 1;
    const bool more = s + 1 < s1;
    v4i next[4];
    if ((F::KS == 1 || s < s1) && ld.works) {
      const uint8_t* st = smem + p * F::kStage + ld.tok_at;
      const uint8_t* sArow = st + r16 * kRowStride + c * 8;
      const uint8_t* sDa = st + F::kTokA + r16 * 16;
      const uint8_t* sTp = st + F::kTokA + F::kTokDa;
      uint8_t* sW = smem + 2 * F::kStage + ld.wave * F::kExpanded;
      const float* sWw = reinterpret_cast<const float*>(sW);
      const v4i hdr =
          *reinterpret_cast<const v4i*>(smem + p * F::kStage + ld.hdr_at + (lane & 31) * 16);
      q4k_stage_scales(hdr, lane & 31, lane >= 32, sW);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      float4 da2;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (b % 2 == 0) set_priority(3 - b / 2);
        if (more) {
          if (b == 0) {
#pragma unroll
            for (int gi = 0; gi < 4; ++gi) next[gi] = ld.nibbles16(s + 1, gi);
          }
#pragma unroll
          for (int v = 0; v < F::kOps; ++v)
            if ((v / 3 * 2 < 7 ? v / 3 * 2 : 7) == b) ld.issue(v, s + 1, p ^ 1);
        }
        uint2 tok = *reinterpret_cast<const uint2*>(sArow + b * 32);
        asm volatile("" : "+v"(tok.x), "+v"(tok.y));  // the steps stay in order
        if (b % 2 == 0) da2 = *reinterpret_cast<const float4*>(sDa + (b >> 1) * F::BM * 16);
        const float2 da = b % 2 == 0 ? make_float2(da2.x, da2.y) : make_float2(da2.z, da2.w);
        const long top = __builtin_bit_cast(long, tok);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t x = (uint32_t)raw[b >> 1][2 * w], y = (uint32_t)raw[b >> 1][2 * w + 1];
          const uint2 wv = b & 1 ? make_uint2((x >> 4) & 0x0F0F0F0Fu, (y >> 4) & 0x0F0F0F0Fu)
                                 : make_uint2(x & 0x0F0F0F0Fu, y & 0x0F0F0F0Fu);
          const v4i D = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, wv), top, bias,
                                                              0, 0, 0);
          const float4 d = *reinterpret_cast<const float4*>(sWw + b * 32 + 16 * w + 4 * c);
          const float ds[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int Dr = D[r];
            acc[w][r] = __builtin_fmaf(__builtin_fmaf(__int_as_float(Dr), da.x, da.y), ds[r], acc[w][r]);
          }
        }
        if (b == 1 || b == 3 || b == 5) {  // a third of term2, as in sums
          const int u = b >> 1;
          const int ia = u == 0 ? 0 : (u == 1 ? 1 - h : 1 + h);
          const int jb = u == 0 ? h : (u == 1 ? 2 * h : 1 - h);
          const v4s tb = *reinterpret_cast<const v4s*>(sTp + (jb * F::BM + r16) * 16 + part);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const v4s wa = *reinterpret_cast<const v4s*>(
                sW + kWDsvBytes + (ia * 32 + 16 * w + r16) * 16 + part);
            acc[w] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(wa, tb, acc[w], 0, 0, 0);
          }
        }
      }
    } else if (more) {
#pragma unroll
      for (int v = 0; v < F::kOps; ++v) ld.issue(v, s + 1, p ^ 1);
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int gi = 0; gi < 4; ++gi) raw[gi] = next[gi];
  }
}

// Out of the lanes' registers: four of a row to 64 bytes (gated: two, the lanes of the gate and the up values
// of one output changing one half of them).
template <int EPI>
__device__ __forceinline__ void store16(const int2* rows, const Args& g, int wt, int lane,
                                        const v4f (&acc)[2], const EpiParam<EPI>& epi) {
  const int c = lane >> 4, pair = rows[lane & 15].x;
  const bool ok = pair >= 0 && wt < (g.N + 31) >> 5;
  auto put = [&](int cols, int j, float a, float b, float d, float e) {
    float* o = g.out + (size_t)pair * cols + j;
    if ((cols & 3) == 0 && j + 3 < cols) {
      *reinterpret_cast<float4*>(o) = make_float4(a, b, d, e);
    } else {
      if (j + 0 < cols) o[0] = a;
      if (j + 1 < cols) o[1] = b;
      if (j + 2 < cols) o[2] = d;
      if (j + 3 < cols) o[3] = e;
    }
  };
  if constexpr (EPI == kEpiGated) {
    const bool low = c < 2;  // has the gate values of both tiles; keeps the first
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float other = __shfl_xor(low ? acc[1][r] : acc[0][r], 32);
      v[r] = activate(low ? acc[0][r] : other, epi.act) * (low ? other : acc[1][r]);
    }
    if (ok) put(epi.F, wt * 16 + (low ? 0 : 8) + 4 * (c & 1), v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = activate(acc[w][r], epi.act);
      if (ok) put(g.N, wt * 32 + 16 * w + 4 * c, v[0], v[1], v[2], v[3]);
    }
  }
}

// Out through a transpose in the wavefront's own 32 x 20 floats of LDS, 16 columns at a time: four lanes
// to a row's 64 bytes. A row's address is its pair's.
template <class F, int TT, int EPI>
__device__ __forceinline__ void store(float* reg, const int2* rows, const Args& g, int wt, int lane,
                                      const v16f (&acc)[TT], const EpiParam<EPI>& epi) {
  const int h = lane >> 5, l32 = lane & 31;
  const bool wt_ok = wt < (g.N + 31) >> 5;
  if constexpr (EPI == kEpiGated) {
    constexpr int TS = 20;
    const int cols = epi.F;
    const int rr = lane >> 2, c4 = lane & 3;  // read-back: rows rr + 16 k, columns 4*c4..+3
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = activate(acc[t][8 * c + r], epi.act) * acc[t][8 * c + 4 + r];
        *reinterpret_cast<float4*>(reg + l32 * TS + 8 * c + 4 * h) =
            make_float4(v[0], v[1], v[2], v[3]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (wt_ok) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = rr + 16 * k;
          const int pair = rows[t * 32 + row].x;
          const int j = wt * 16 + 4 * c4;
          if (pair < 0) continue;
          const float4 v = *reinterpret_cast<const float4*>(reg + row * TS + 4 * c4);
          float* o = g.out + (size_t)pair * cols + j;
          if ((cols & 3) == 0 && j + 3 < cols) {
            *reinterpret_cast<float4*>(o) = v;
          } else {
            if (j + 0 < cols) o[0] = v.x;
            if (j + 1 < cols) o[1] = v.y;
            if (j + 2 < cols) o[2] = v.z;
            if (j + 3 < cols) o[3] = v.w;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    constexpr int TS = 20;
    const int rr = lane >> 2, c4 = lane & 3;  // read-back: rows rr + 16 k, columns 4*c4..+3
    const int N = g.N;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // 16 of the 32 columns
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
          const int r = 8 * half + 4 * gi;
          *reinterpret_cast<float4*>(reg + l32 * TS + 8 * gi + 4 * h) =
              make_float4(acc[t][r], acc[t][r + 1], acc[t][r + 2], acc[t][r + 3]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (wt_ok) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int row = rr + 16 * k;
            const int pair = rows[t * 32 + row].x;
            const int j = wt * 32 + 16 * half + 4 * c4;
            if (pair < 0) continue;
            float4 v = *reinterpret_cast<const float4*>(reg + row * TS + 4 * c4);
            if (epi.act != kActNone) {
              v.x = activate(v.x, epi.act); v.y = activate(v.y, epi.act);
              v.z = activate(v.z, epi.act); v.w = activate(v.w, epi.act);
            }
            float* o = g.out + (size_t)pair * N + j;
            if ((N & 3) == 0 && j + 3 < N) {
              *reinterpret_cast<float4*>(o) = v;
            } else {
              if (j + 0 < N) o[0] = v.x;
              if (j + 1 < N) o[1] = v.y;
              if (j + 2 < N) o[2] = v.z;
              if (j + 3 < N) o[3] = v.w;
            }
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
}

// A tile with its rows found, in parts of 32 rows or (FEW) as one of 16: two copies of all that follows, since
// the compiler keeps the registers of code that both would share through either.
template <class F, int EPI, bool FEW>
__device__ __forceinline__ void tile(uint8_t* smem, const Args& g, const Pick& t, int2 row,
                                     const EpiParam<EPI>& epi) {
  const int tid = threadIdx.x;
  int2* rows = reinterpret_cast<int2*>(smem + F::kRowsAt);
  Loads<F> ld;
  ld.init(smem, g);
  ld.aim(g, t);
  const int nsb = g.K >> 8;
  const int ks = F::KS == 1 ? 0 : ld.wave / F::CW;
  const int s0 = F::KS == 1 ? 0 : ks * nsb / F::KS, s1 = F::KS == 1 ? nsb : (ks + 1) * nsb / F::KS;
  const int steps = F::KS == 1 ? nsb : (nsb + F::KS - 1) / F::KS;  // the longest range's
  const bool any = F::KS == 1 || s0 < s1;
  v4i raw[4];
  if (any) {  // the weights while the rows are on their way
#pragma unroll
    for (int gi = 0; gi < 4; ++gi) raw[gi] = FEW ? ld.nibbles16(s0, gi) : ld.nibbles(s0, gi);
  }
  if (tid < F::BM) rows[tid] = row;
  __syncthreads();
  ld.aim(g, rows);
  if (any) {
#pragma unroll
    for (int v = 0; v < F::kOps; ++v) ld.issue(v, s0, 0);
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  // The other ranges' sums, [range][wavefront][register][lane], added in the order of the ranges; whether
  // this wavefront has them then.
  auto join = [&](auto& acc) -> bool {
    constexpr int V = sizeof(acc[0]) / 4, N = sizeof(acc) / 4;
    if constexpr (F::KS > 1) {
      static_assert((F::KS - 1) * F::CW * N * 256 <= 2 * F::kStage, "LDS of the sums");
      float* red = reinterpret_cast<float*>(smem) + ld.lane;
      if (ks > 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) red[(((ks - 1) * F::CW + ld.cw) * N + r) * 64] = acc[r / V][r % V];
      }
      __syncthreads();
      if (ks > 0) return false;
#pragma unroll
      for (int o = 0; o < F::KS - 1; ++o)
#pragma unroll
        for (int r = 0; r < N; ++r) acc[r / V][r % V] += red[((o * F::CW + ld.cw) * N + r) * 64];
    }
    return true;
  };
  const int wt = t.tn * F::CW + ld.cw;
  if constexpr (FEW) {
    v4f acc[2];
    sums16<F>(smem, ld, s0, s1, steps, raw, acc);
    if (join(acc)) store16<EPI>(rows, g, wt, ld.lane, acc, epi);
  } else {
    auto run = [&](auto parts) {
      constexpr int TT = decltype(parts)::value;
      v16f acc[TT];
      sums<F, TT>(smem, ld, s0, s1, steps, raw, acc);
      if (!join(acc)) return;
      // through the wavefront's region of weight scales
      store<F, TT, EPI>(reinterpret_cast<float*>(smem + 2 * F::kStage + ld.wave * F::kExpanded), rows,
                        g, wt, ld.lane, acc, epi);
    };
    using std::integral_constant;
    if constexpr (F::TMAX == 4) {
      if (ld.parts == 4) return run(integral_constant<int, 4>{});
      if (ld.parts == 3) return run(integral_constant<int, 3>{});
      if (ld.parts == 2) return run(integral_constant<int, 2>{});
    }
    static_assert(F::TMAX == 1 || F::TMAX == 4, "the numbers of parts");
    run(integral_constant<int, 1>{});
  }
}

template <class F, int EPI>
__global__ __launch_bounds__(F::NW * 64, F::WAVES) void grouped_kernel(Args g, EpiParam<EPI> epi) {
  extern __shared__ __align__(16) uint8_t smem[];
  static_assert(F::BM <= 64 * F::NW, "a work-item per row");
  const Pick t = find_tile<F>(*reinterpret_cast<SearchLds*>(smem), g);
  if (t.rows <= 0) return;
  int2 row = make_int2(-1, 0);
  if ((int)threadIdx.x < F::BM) row = load_row<F>(g, t);
  if constexpr (F::TMAX == 1) {
    if (t.rows <= 16) return tile<F, EPI, true>(smem, g, t, row, epi);
  }
  tile<F, EPI, false>(smem, g, t, row, epi);
}

template <class F, int EPI>
hipError_t launch_t(const void* q8, const int* groups, const void* w, float* out,
                    const GroupedShape& g, const Epilogue& epi, int64_t cus, hipStream_t s) {
  const uint8_t* base = static_cast<const uint8_t*>(q8);
  auto kern = grouped_kernel<F, EPI>;
  if (F::kLds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, F::kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t gn = ((g.N + 31) / 32 + F::CW - 1) / F::CW;
  const int64_t most = g.P / F::BM + (g.E < g.P ? g.E : g.P);
  const int64_t slots = std::max<int64_t>(1, cus / 8);
  const int64_t grid = ((most * gn + 7) / 8 + (F::kTail ? slots : 0)) * 8;
  const Args a{reinterpret_cast<const int8_t*>(base),
               reinterpret_cast<const float*>(base + q8_planes_offset(g.q_rows, g.K)),
               reinterpret_cast<const uint16_t*>(base + q8_pieces_offset(g.q_rows, g.K)),
               groups, static_cast<const uint8_t*>(w), out, (int)g.P, (int)g.E, (int)g.N, (int)g.K,
               (int)g.q_rows, (int)g.per_row, (int)gn, (int)GroupLayout{g.P, g.E}.order(),
               (int)most, (int)slots};
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * F::NW), (size_t)F::kLds, s, a,
                     epi_param<EPI>(epi));
  return hipGetLastError();
}

// The forms of the kernel.
using Wide = Form<4, 8, 1, 2>;   // 128 rows x 256 weight rows, one workgroup to a compute unit
using Narrow = Form<1, 4, 1, 4>; // 32 x 128, four
using Split2 = Form<1, 4, 2, 4>; // 32 x 128, K in two ranges, two
using Split4 = Form<1, 4, 4, 4>; // 32 x 128, K in four ranges, one

template <int EPI>
hipError_t launch_epi(const void* q8, const int* groups, const void* w, float* out,
                      const GroupedShape& g, const Epilogue& epi, int64_t cus, hipStream_t s) {
  switch (grouped_form(g, cus)) {
    case kGroupedNarrow: return launch_t<Narrow, EPI>(q8, groups, w, out, g, epi, cus, s);
    case kGroupedSplit2: return launch_t<Split2, EPI>(q8, groups, w, out, g, epi, cus, s);
    case kGroupedSplit4: return launch_t<Split4, EPI>(q8, groups, w, out, g, epi, cus, s);
    default: return launch_t<Wide, EPI>(q8, groups, w, out, g, epi, cus, s);
  }
}

}  // namespace

GroupedForm grouped_form(const GroupedShape& g, int64_t compute_units) {
  const double cus = (double)compute_units, nsb = (double)(g.K / 256);
  const double ntiles = (double)((g.N + 31) / 32);
  // experts that P evenly drawn pairs name, and the tiles of 32 and 128 rows they make
  const double E = (double)g.E, P = (double)g.P;
  const double used = E * (1.0 - std::pow(1.0 - 1.0 / E, P)), r = P / used;
  const double t32 = used * std::max(1.0, r / 32.0 + 0.5);
  const double t128 = used * std::max(1.0, r / 128.0 + 0.5);
  // Rounds of a grid over the device: one, or, the last one being partly empty, half a round more. An expected
  // grid just within one round can need two by the ids: 300 tokens, 2 of 8, 4096 -> 1376 in four ranges make 21
  // to 23 tiles on 23 of 24 draws, 27 us in a graph, and 24 on one, 264 workgroups, 41 us.
  auto rounds = [](double grid, double slots) { return grid <= slots ? 1.0 : grid / slots + 0.5; };
  // per super-block of a 32-row tile with u wavefronts to a SIMD
  auto us = [](double u) {
    return u <= 2.0 ? 1.5 + 0.3 * std::max(u, 1.0) : u <= 4.0 ? 2.1 + 0.55 * (u - 2.0) : 3.2;
  };
  const double wide = t128 * std::ceil(ntiles / 8.0), narrow = t32 * std::ceil(ntiles / 4.0);
  const double load = narrow / cus;
  // What a form takes: rounds of its grid, times a workgroup's microseconds per super-block and its fixed ones
  // (search, gather, first loads, store). Measured in every form (us, wide / narrow / two ranges of K / four;
  // graph replays, quantization included), the choice being the best one or as said:
  //   gated, 64 experts, 8 slots, D = 2048, F = 1024:  100 tokens 56 / 49 / 53 / 65, 512 111 / 99 / 106 /
  //     142, 2048 254 / 286 / 307 / 407 (chosen: 258)
  //   gated, 8 experts, 2 slots, D = 4096, F = 5504:   80 tokens 88 / 67 / 74 / 85, 500 203 / 204 / 212 / 248
  //   gated, 16 experts, 2 slots, 2048, 1024:          20 tokens 24 / 22 / 18 / 18, 4000 (D = 1024) 94 / 92 /
  //     109 / 153
  //   plain, 8 experts, 300 tokens of 2, 4096 -> 1376: 87 / 43 / 32 / 28
  //   down, 8 experts, 2 slots, 5632 -> 4096:          24 tokens 51 / 47 / 34 / 33, 80 67 / 57 / 46 / 52,
  //     500 133 / 138 / 138 / 144 (chosen: 131)
  //   down, 64 experts, 8 slots, 1024 -> 2048:         100 tokens 41 / 38 / 41 / 52, 2048 206 / 220 / 246 /
  //     335 (chosen: narrow, the furthest of 36 shapes from their best, 7 %; the others are within 3 %)
  const double cost[4] = {
      rounds(wide, cus) * (nsb * (1.0 + 0.95 * t32 / t128) + 13.0),
      rounds(narrow, 4.0 * cus) * (nsb * us(load) + 5.0),
      rounds(narrow, 2.0 * cus) * (std::ceil(nsb / 2.0) * us(2.0 * load) + 6.0),
      rounds(narrow, cus) * (std::ceil(nsb / 4.0) * 3.5 + 7.0)};
  // Dividing K gains nothing where the narrow tiles fill the device many times over; the bound keeps the
  // split forms' grids (at most 2.6 times `narrow`, workgroups of up to 1024) far below 2^32 work-items.
  const int forms = narrow <= 64.0 * cus ? 4 : 2;
  return (GroupedForm)(std::min_element(cost, cost + forms) - cost);
}

int64_t grouped_lds_bytes(GroupedForm f) {
  return f == kGroupedNarrow   ? Narrow::kLds
         : f == kGroupedSplit2 ? Split2::kLds
         : f == kGroupedSplit4 ? Split4::kLds
                               : Wide::kLds;
}

hipError_t launch_grouped(const void* q8, const int* groups, const void* w, float* out,
                          const GroupedShape& g, const Epilogue& epi, int64_t cus, hipStream_t s) {
  return epi.kind == kEpiGated ? launch_epi<kEpiGated>(q8, groups, w, out, g, epi, cus, s)
                               : launch_epi<kEpiAct>(q8, groups, w, out, g, epi, cus, s);
}

}  // namespace mmq
