// The q4_K x q8_1 product grouped by expert: out[p] = act(x[src(p)] W(e)^T), or its gated form, for
// every pair p of the groups with an expert e, the rows of one expert being one ragged matrix.
//
// The arithmetic is the tile of mmq_gemm.hip, per element the same operations in the same order (its
// comment has the mathematics: one int8 MFMA per 32-block, two FMAs per element to rescale it, term2
// on the bf16 unit, three instructions per super-block), so one expert that has all rows gives the
// plain product's bits. It is bound as that kernel is, by the rescale's vector instructions. What
// differs is which rows a workgroup has and how they get into LDS:
//
// - The host knows the pairs, not how they fall on the experts. The grid covers the most tiles that
//   they can form (P / BM + min(E, P) for tiles of BM rows); a workgroup finds its expert and rows
//   from the offsets of the groups, one work-item per expert and one prefix sum, and ends at once
//   where there is no such tile.
// - An expert's rows are cut into tiles of 32 TT rows, the last one of the 32-row parts it needs: the
//   tile's code exists for 1 .. TT parts and a workgroup branches to its own, so a tile of few rows
//   does not pay for the rescale of many.
// - The rows are gathered by the loads into LDS: each lane's address has its row's place in the q8
//   buffer, taken from the groups once per workgroup. quantize_q8_1's (da, nda) plane is block-major
//   for contiguous rows; here it is row-major, 16 bytes holding two blocks of a row, and is staged as
//   [4 pairs of blocks][BM] of 16 bytes. (Its 8-byte reads then meet two ways in the LDS banks, one
//   read per 33 vector instructions.) Tokens are quantized once, not once per slot.
// - Workgroups go to the XCDs in turn. Each XCD gets a contiguous range of the tiles in the order
//   (weight-tile group, expert, rows), so the row tiles that share weights run on one L2.
#include "epilogue.h"
#include "grouped_internal.h"
#include "mmq_device.h"

namespace mmq {
namespace {

__device__ __forceinline__ void set_priority(int p) {
  if (p >= 3) __builtin_amdgcn_s_setprio(3);
  else if (p == 2) __builtin_amdgcn_s_setprio(2);
  else if (p == 1) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

constexpr int kNW = 8;  // wavefronts of a workgroup, one 32-row weight tile each

// What a tile needs besides its rows.
struct TileArgs {
  const int8_t* qs;
  const float* da;
  const uint16_t* pieces;
  const uint8_t* w;   // the expert's records
  float* out;
  int q_rows, per_row, N, K, tn;
};

// One tile of 32 TT rows. rows[i] is the pair of row i, -1 past the tile's last row.
template <int TT, int EPI>
__device__ __forceinline__ void tile(uint8_t* smem, const int* rows, const TileArgs& g,
                                     const EpiParam<EPI>& epi) {
  constexpr int NW = kNW;
  constexpr int BM = 32 * TT;
  constexpr int NS = 8 * TT;                      // (block, token tile) steps per super-block
  constexpr int A_BYTES = BM * kRowStride;        // token tile
  constexpr int DA_BYTES = BM * 64;               // (da, nb) pairs [4][BM][2 blocks][2]
  constexpr int TP_BYTES = BM * 48;               // token pieces of da*sa [3][BM][8]
  constexpr int W_BYTES = kWDsvBytes + kWPieceBytes + kRepHdrBytes;
  constexpr int STAGE = A_BYTES + DA_BYTES + TP_BYTES + NW * W_BYTES;
  static_assert(STAGE == TileShape{TT, NW}.stage_bytes(), "LDS stage layout");
  constexpr int A_SLOTS = BM * (kRowStride / 16);  // 16-byte slots of the token tile
  constexpr int A_DMA = (A_SLOTS + 63) / 64;       // wavefront-wide DMA instructions
  constexpr int A_PER_WAVE = (A_DMA + NW - 1) / NW;
  constexpr int DA_SLOTS = 4 * BM;
  constexpr int DA_DMA = (DA_SLOTS + 63) / 64;
  constexpr int DA_PER_WAVE = (DA_DMA + NW - 1) / NW;
  constexpr int TP_SLOTS = 3 * BM;
  constexpr int TP_DMA = (TP_SLOTS + 63) / 64;
  constexpr int TP_PER_WAVE = (TP_DMA + NW - 1) / NW;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5;
  const int l32 = lane & 31;

  const int N = g.N, K = g.K;
  const int ntiles = (N + 31) >> 5;
  const int wt_raw = g.tn * NW + wave;
  const bool wt_ok = wt_raw < ntiles;
  const int wt = wt_ok ? wt_raw : ntiles - 1;  // idle wavefronts still stage and sync
  const int nsb = K >> 8;
  const uint32_t M = (uint32_t)g.q_rows;
  const uint32_t q_bytes = M * (uint32_t)K;
  const uint32_t da_bytes = q_bytes >> 2;
  const uint32_t tp_bytes = M * (uint32_t)nsb * 48u;
  const v4i rq = make_rsrc_sgpr(g.qs, q_bytes);
  const v4i rda = make_rsrc_sgpr(g.da, da_bytes);
  const v4i rtp = make_rsrc_sgpr(g.pieces, tp_bytes);
  const uint8_t* wtile = g.w + (size_t)wt * nsb * kRepTileBytes;
  const v4i rwd = make_rsrc_sgpr(wtile, (uint32_t)nsb * kRepTileBytes);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wtile, (uint32_t)nsb * kRepTileBytes);

  // The row of the q8 buffer of the tile's row r; none (the buffers' end, which reads zero) past it.
  auto src_of = [&](int r) -> uint32_t {
    const int p = rows[r];
    return p < 0 ? M : (uint32_t)p / (uint32_t)g.per_row;
  };
  // Token-tile DMA slots of this lane: slot q = 64*k + lane holds chunk q % 17 of row q / 17;
  // chunk 16 is the row's padding and reads past the end (zero), as do rows past the last.
  uint32_t a_off[A_PER_WAVE];
  bool a_act[A_PER_WAVE];
#pragma unroll
  for (int j = 0; j < A_PER_WAVE; ++j) {
    const int k = wave + j * NW;
    const int q = k * 64 + lane;
    const int row = q / 17, c = q - row * 17;
    a_act[j] = k < A_DMA && q < A_SLOTS;
    const uint32_t src = a_act[j] ? src_of(row) : M;
    a_off[j] = c < 16 && src < M ? src * (uint32_t)K + c * 16 : q_bytes;
  }
  // (da, nb): slot q holds pair of blocks q / BM of row q % BM; 64 bytes per row and super-block.
  uint32_t da_off[DA_PER_WAVE];
  bool da_act[DA_PER_WAVE];
#pragma unroll
  for (int j = 0; j < DA_PER_WAVE; ++j) {
    const int k = wave + j * NW;
    const int q = k * 64 + lane;
    const int bp = q / BM, r = q - bp * BM;
    da_act[j] = k < DA_DMA && q < DA_SLOTS;
    const uint32_t src = da_act[j] ? src_of(r) : M;
    da_off[j] = src < M ? src * ((uint32_t)K >> 2) + bp * 16 : da_bytes;
  }
  // Token pieces: slot q holds piece q / BM of row q % BM; [super-block][piece][M][8] in memory. A
  // row past the last starts at the end of the plane, and stays past it with every super-block.
  uint32_t tp_off[TP_PER_WAVE];
  bool tp_act[TP_PER_WAVE];
#pragma unroll
  for (int j = 0; j < TP_PER_WAVE; ++j) {
    const int k = wave + j * NW;
    const int q = k * 64 + lane;
    const int pc = q / BM, r = q - pc * BM;
    tp_act[j] = k < TP_DMA && q < TP_SLOTS;
    const uint32_t src = tp_act[j] ? src_of(r) : M;
    tp_off[j] = src < M ? ((uint32_t)pc * M + src) * 16u : tp_bytes;
  }
  // What a stage loads into LDS, as NOPS - 1 DMA instructions of this wavefront, and, as the last
  // op, its last 16 bytes of nibbles into registers; spread over the previous super-block's steps as
  // in mmq_gemm.hip.
  constexpr int NOPS = A_PER_WAVE + DA_PER_WAVE + TP_PER_WAVE + 2;
  auto op_step = [](int v) { return ((v / 3) * 2 * TT < NS - 1) ? (v / 3) * 2 * TT : NS - 1; };
  auto load_nib = [&](int s, int gi) -> v4i {
    return buf_load16(rw, (uint32_t)s * kRepTileBytes + gi * 1024 + lane * 16);
  };
  const uint32_t lds0 = lds_addr(smem);
  auto issue_op = [&](int v, int s, int p, v4i& nib3) {
    const uint32_t st = lds0 + (uint32_t)(p * STAGE);
    if (v < A_PER_WAVE) {
      const int k = wave + v * NW;
      if (k < A_DMA && a_act[v]) dma16(rq, st + k * 1024, a_off[v] + (uint32_t)s * 256);
      return;
    }
    v -= A_PER_WAVE;
    if (v < DA_PER_WAVE) {
      const int k = wave + v * NW;
      if (k < DA_DMA && da_act[v])
        dma16(rda, st + A_BYTES + k * 1024, da_off[v] + (uint32_t)s * 64);
      return;
    }
    v -= DA_PER_WAVE;
    if (v < TP_PER_WAVE) {
      const int k = wave + v * NW;
      if (k < TP_DMA && tp_act[v])
        dma16(rtp, st + A_BYTES + DA_BYTES + k * 1024, tp_off[v] + (uint32_t)s * 3u * M * 16u);
      return;
    }
    v -= TP_PER_WAVE;
    if (v < 1) {
      const uint32_t sw = st + A_BYTES + DA_BYTES + TP_BYTES + wave * W_BYTES;
      if (lane < 32)
        dma16(rwd, sw + kWDsvBytes + kWPieceBytes,
              (uint32_t)s * kRepTileBytes + kRepNibBytes + lane * 16);
      return;
    }
    nib3 = load_nib(s, 3);
  };

  v16i bias;
#pragma unroll
  for (int r = 0; r < 16; ++r) bias[r] = kBiasBits;
  asm volatile("" : "+v"(bias));  // stays in vector registers, as in mmq_gemm.hip
  v16f acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.0f;

  // The nibbles of the next stage: in place as they are used up, or (one token tile: a super-block is
  // too short for that) all at the first step, through a second set. As in mmq_gemm.hip.
  constexpr bool ENIB = TT == 1;
  v4i raw[4], nib3, rawB[ENIB ? 4 : 1];
#pragma unroll
  for (int v = 0; v < NOPS - (ENIB ? 1 : 0); ++v) issue_op(v, 0, 0, nib3);
#pragma unroll
  for (int gi = 0; gi < (ENIB ? 4 : 3); ++gi) raw[gi] = load_nib(0, gi);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  for (int s = 0; s < nsb; ++s) {
    const int p = s & 1;
    if constexpr (!ENIB) raw[3] = nib3;
    const bool more = s + 1 < nsb;

    const uint8_t* st = smem + p * STAGE;
    const uint8_t* sArow = st + l32 * kRowStride + h * 16;
    const uint8_t* sDa = st + A_BYTES;
    const uint8_t* sTp = st + A_BYTES + DA_BYTES;
    const uint8_t* sW = st + A_BYTES + DA_BYTES + TP_BYTES + wave * W_BYTES;
    const float* sWw = reinterpret_cast<const float*>(sW);
    auto expand_scales = [&]() {
      uint8_t* sWm = smem + p * STAGE + A_BYTES + DA_BYTES + TP_BYTES + wave * W_BYTES;
      const v4i hdr =
          *reinterpret_cast<const v4i*>(sWm + kWDsvBytes + kWPieceBytes + l32 * 16);
      q4k_stage_scales(hdr, l32, h != 0, sWm);
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
    auto da_of = [&](int n) -> float2 {
      const int b = n / TT, t = n % TT;
      return *reinterpret_cast<const float2*>(sDa + ((b >> 1) * BM + t * 32 + l32) * 16 +
                                              (b & 1) * 8);
    };
    auto dsv_of = [&](int b, float (&d)[16]) {
#pragma unroll
      for (int gi = 0; gi < 4; ++gi) {
        const float4 a = *reinterpret_cast<const float4*>(sWw + b * 32 + 8 * gi + 4 * h);
        d[4 * gi + 0] = a.x; d[4 * gi + 1] = a.y; d[4 * gi + 2] = a.z; d[4 * gi + 3] = a.w;
      }
    };

    // Entering step n = b*TT + t: D(n) has been issued, the token operand of step n+1 and da of
    // step n are in registers; dsv[b & 1] holds block b's weight scales.
    v16i Dn = __builtin_amdgcn_mfma_i32_32x32x32_i8(wop_of(0), top_of(0), bias, 0, 0, 0);
    asm volatile("" : "+v"(Dn));  // issued here, not sunk below the expansion
    v4i tnext = top_of(1 % NS);
    float2 da = da_of(0);
    expand_scales();
    float dsv[2][16];
    dsv_of(0, dsv[0]);
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int b = n / TT, t = n % TT;
      if (n % 2 == 0) set_priority(3 - (n % 8) / 2);  // the pair of a SIMD keeps step
      if (more) {
        if constexpr (ENIB) {
          if (n == 0) {
#pragma unroll
            for (int gi = 0; gi < 4; ++gi) rawB[gi] = load_nib(s + 1, gi);
          }
#pragma unroll
          for (int v = 0; v < NOPS - 1; ++v)
            if (op_step(v) == n) issue_op(v, s + 1, p ^ 1, nib3);
        } else {
#pragma unroll
          for (int v = 0; v < NOPS; ++v)
            if (op_step(v) == n) issue_op(v, s + 1, p ^ 1, nib3);
#pragma unroll
          for (int gi = 0; gi < 3; ++gi)
            if (n == (2 * gi + 2) * TT) raw[gi] = load_nib(s + 1, gi);
        }
      }
      const v16i D = Dn;
      const float2 dac = da;  // (da, nb)
      if (n + 1 < NS) {
        Dn = __builtin_amdgcn_mfma_i32_32x32x32_i8(wop_of((n + 1) / TT), tnext, bias, 0, 0, 0);
        da = da_of(n + 1);
      }
      if (n + 2 < NS) tnext = top_of(n + 2);
      if (t == 0 && b + 1 < 8) dsv_of(b + 1, dsv[(b + 1) & 1]);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float y = __builtin_fmaf(__int_as_float(D[r]), dac.x, dac.y);
        acc[t][r] = __builtin_fmaf(y, dsv[b & 1][r], acc[t][r]);
      }
      if (b == 1 || b == 3 || b == 5) {  // a third of term2, the piece pairs of mmq_gemm.hip
        const int u = b >> 1;
        const int ia = u == 0 ? 0 : (u == 1 ? 1 - h : 1 + h);
        const int jb = u == 0 ? h : (u == 1 ? 2 * h : 1 - h);
        const v8bf wa = *reinterpret_cast<const v8bf*>(sW + kWDsvBytes + (ia * 32 + l32) * 16);
        const v8bf tb = *reinterpret_cast<const v8bf*>(sTp + (jb * BM + t * 32 + l32) * 16);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa, tb, acc[t], 0, 0, 0);
      }
    }

    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_s_waitcnt(0);  // this wavefront's stage s+1 loads have landed
    __syncthreads();                // ... and everyone's; stage s is no longer read
    if constexpr (ENIB) {
#pragma unroll
      for (int gi = 0; gi < 4; ++gi) raw[gi] = rawB[gi];
    }
  }

  // Out through the wavefront's own LDS regions, as in mmq_gemm.hip; a row's address is its pair's.
  float* out = g.out;
  if constexpr (EPI == kEpiGated) {
    constexpr int TS = 20;
    const int F = epi.F;
    const int rr = lane >> 2, c4 = lane & 3;  // read-back: rows rr + 16 k, columns 4*c4..+3
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float* reg = reinterpret_cast<float*>(smem) + ((t & 1) * NW + wave) * (32 * TS);
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
          const int pair = rows[t * 32 + row];
          const int j = wt * 16 + 4 * c4;
          if (pair < 0) continue;
          const float4 v = *reinterpret_cast<const float4*>(reg + row * TS + 4 * c4);
          float* o = out + (size_t)pair * F + j;
          if ((F & 3) == 0 && j + 3 < F) {
            *reinterpret_cast<float4*>(o) = v;
          } else {
            if (j + 0 < F) o[0] = v.x;
            if (j + 1 < F) o[1] = v.y;
            if (j + 2 < F) o[2] = v.z;
            if (j + 3 < F) o[3] = v.w;
          }
        }
      }
    }
  } else {
    constexpr int TS = 36;
    const int rr = lane >> 3, c4 = lane & 7;  // read-back: rows rr + 8 k, columns 4*c4..+3
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float* reg = reinterpret_cast<float*>(smem) + ((t & 1) * NW + wave) * (32 * TS);
#pragma unroll
      for (int gi = 0; gi < 4; ++gi)
        *reinterpret_cast<float4*>(reg + l32 * TS + 8 * gi + 4 * h) = make_float4(
            acc[t][4 * gi], acc[t][4 * gi + 1], acc[t][4 * gi + 2], acc[t][4 * gi + 3]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (wt_ok) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = rr + 8 * k;
          const int pair = rows[t * 32 + row];
          const int j = wt * 32 + 4 * c4;
          if (pair < 0) continue;
          float4 v = *reinterpret_cast<const float4*>(reg + row * TS + 4 * c4);
          if (epi.act != kActNone) {
            v.x = activate(v.x, epi.act); v.y = activate(v.y, epi.act);
            v.z = activate(v.z, epi.act); v.w = activate(v.w, epi.act);
          }
          float* o = out + (size_t)pair * N + j;
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
    }
  }
}

// Which tile a workgroup has: 32-row parts of expert e, from its row `first` of the order on.
struct Pick {
  int expert, first, rows, tn;
};

// LDS of the search, over the stages (which are not in use yet).
struct SearchLds {
  int wave_tiles[kNW];
  Pick pick;
};

// Work-item e looks at expert e. The offsets are only used inside [0, P], so that groups of nonsense
// select nonsense rows of this product and no others.
template <int TMAX>
__device__ __forceinline__ Pick find_tile(SearchLds& sh, const int* __restrict__ groups, int P,
                                          int E, int gn, int most) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int lo = 0, n = 0;
  if (tid < E) {
    lo = min(max(groups[tid], 0), P);
    n = min(max(groups[tid + 1], lo), P) - lo;
  }
  const int mine = (n + 32 * TMAX - 1) / (32 * TMAX);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) sh.wave_tiles[wave] = incl;
  if (tid == 0) sh.pick.rows = 0;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kNW; ++w) {
    const int v = sh.wave_tiles[w];
    if (w < wave) before += v;
    all += v;
  }
  all = min(all, most);  // what the grid covers (offsets of nonsense may ask for more)
  // tiles in the order (weight-tile group, rows), one contiguous range per XCD
  const unsigned total = (unsigned)all * (unsigned)gn;
  const unsigned per_xcd = (total + 7u) >> 3;
  const unsigned k = blockIdx.x >> 3;
  const unsigned idx = (blockIdx.x & 7u) * per_xcd + k;
  if (k < per_xcd && idx < total) {
    const int tn = (int)(idx / (unsigned)all);
    const int u = (int)(idx - (unsigned)tn * (unsigned)all) - (before + incl - mine);
    if (u >= 0 && u < mine)
      sh.pick = Pick{tid, lo + u * 32 * TMAX, min(n - u * 32 * TMAX, 32 * TMAX), tn};
  }
  __syncthreads();
  const Pick p = sh.pick;
  return Pick{__builtin_amdgcn_readfirstlane(p.expert), __builtin_amdgcn_readfirstlane(p.first),
              __builtin_amdgcn_readfirstlane(p.rows), __builtin_amdgcn_readfirstlane(p.tn)};
}

template <int TMAX, int EPI>
__global__ __launch_bounds__(kNW * 64, 1) void grouped_kernel(
    const int8_t* __restrict__ qs, const float* __restrict__ da, const uint16_t* __restrict__ pieces,
    const int* __restrict__ groups, const uint8_t* __restrict__ w, float* __restrict__ out, int P,
    int E, int N, int K, int q_rows, int per_row, int gn, int most, int order_at, EpiParam<EPI> epi) {
  constexpr TileShape ts{TMAX, kNW};
  extern __shared__ __align__(16) uint8_t smem[];
  int* rows = reinterpret_cast<int*>(smem + ts.lds_bytes());
  const Pick pick = find_tile<TMAX>(*reinterpret_cast<SearchLds*>(smem), groups, P, E, gn, most);
  if (pick.rows <= 0) return;
  const int tid = threadIdx.x;
  if (tid < 32 * TMAX) {
    const int p = tid < pick.rows ? groups[order_at + pick.first + tid] : -1;
    rows[tid] = p < P ? p : -1;
  }
  __syncthreads();
  const size_t matrix = (size_t)((N + 31) >> 5) * (size_t)(K >> 8) * kRepTileBytes;
  const TileArgs g{qs, da, pieces, w + (size_t)pick.expert * matrix, out, q_rows, per_row, N, K,
                   pick.tn};
  const int parts = (pick.rows + 31) >> 5;
  if constexpr (TMAX >= 4) {
    if (parts == 4) return tile<4, EPI>(smem, rows, g, epi);
    if (parts == 3) return tile<3, EPI>(smem, rows, g, epi);
  }
  if constexpr (TMAX >= 2) {
    if (parts == 2) return tile<2, EPI>(smem, rows, g, epi);
  }
  tile<1, EPI>(smem, rows, g, epi);
}

constexpr int64_t lds_bytes(int tmax) {
  return TileShape{tmax, kNW}.lds_bytes() + 32 * tmax * (int64_t)sizeof(int);
}

// 32-row parts of the largest tile, and the most tiles that the pairs can form.
int tile_parts(const GroupedShape&) { return 4; }
int64_t most_tiles(const GroupedShape& g) {
  return g.P / (32 * tile_parts(g)) + (g.E < g.P ? g.E : g.P);
}

template <int TMAX, int EPI>
hipError_t launch_t(const void* q8, const int* groups, const void* w, float* out,
                    const GroupedShape& g, const Epilogue& epi, hipStream_t s) {
  const uint8_t* base = static_cast<const uint8_t*>(q8);
  auto kern = grouped_kernel<TMAX, EPI>;
  constexpr int64_t lds = lds_bytes(TMAX);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const int64_t gn = (g.N + 32 * kNW - 1) / (32 * kNW);
  hipLaunchKernelGGL(kern, dim3((unsigned)grouped_grid(g)), dim3(64 * kNW), (size_t)lds, s,
                     reinterpret_cast<const int8_t*>(base),
                     reinterpret_cast<const float*>(base + q8_planes_offset(g.q_rows, g.K)),
                     reinterpret_cast<const uint16_t*>(base + q8_pieces_offset(g.q_rows, g.K)),
                     groups, static_cast<const uint8_t*>(w), out, (int)g.P, (int)g.E, (int)g.N,
                     (int)g.K, (int)g.q_rows, (int)g.per_row, (int)gn, (int)most_tiles(g),
                     (int)GroupLayout{g.P, g.E}.order(), epi_param<EPI>(epi));
  return hipGetLastError();
}

template <int EPI>
hipError_t launch_epi(const void* q8, const int* groups, const void* w, float* out,
                      const GroupedShape& g, const Epilogue& epi, hipStream_t s) {
  return launch_t<4, EPI>(q8, groups, w, out, g, epi, s);
}

}  // namespace

int64_t grouped_grid(const GroupedShape& g) {
  const int64_t gn = (g.N + 32 * kNW - 1) / (32 * kNW);
  return (most_tiles(g) * gn + 7) / 8 * 8;
}
int64_t grouped_lds_bytes(const GroupedShape& g) { return lds_bytes(tile_parts(g)); }

hipError_t launch_grouped(const void* q8, const int* groups, const void* w, float* out,
                          const GroupedShape& g, const Epilogue& epi, hipStream_t s) {
  return epi.kind == kEpiGated ? launch_epi<kEpiGated>(q8, groups, w, out, g, epi, s)
                               : launch_epi<kEpiAct>(q8, groups, w, out, g, epi, s);
}

}  // namespace mmq
