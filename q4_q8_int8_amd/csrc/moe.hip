// The two products of a mixture-of-experts layer for a few tokens, over q4_K weights and q8_1
// activations, each reading a used expert's weights once per group of its columns.
//
// With p = t * k + s the pair (token t, slot s), e(p) its expert:
//   gated   H[p] = act(x[t] Wg(e)^T) * (x[t] Wu(e)^T)        (pair records, epilogue.h)
//   down    out[t] = sum over the slots s of weight[p] * (H[p] Wd(e)^T) + residual[t]
// The plan (moe_route.hip) lists the used experts in increasing order, each with its pairs, so a
// workgroup finds the rows of its product, the expert's columns below, in one list.
//
// Both are bound by reading the used experts' weights (4.5 bits each; nothing else is of their
// size): 16 tokens, 2 of 8 experts (D = 4096, F = 11008, 8 experts used) read their 406 MB of gate and
// up weights in 89 us, 4.5 TB/s (graph replays over six copies, quantization included), a large device
// copy moving 5.2. A wavefront's product is a DotWave (moe_dot.h, a few columns) or a MfmaWave
// (moe_mfma.h, up to 16). An expert with more columns than the form takes (gated: 16, with one token 1;
// down: 16, 8, 4, 3 or 1) is worked through in groups, its weights read again for each, in part from
// the caches (the gated product of 64 tokens, 2 of 8, reads 613 MB for 406 MB of weights). Sums are
// float32 in a fixed order: no atomics, the same bits on every call.
//
// The host does not know the plan, so it chooses the form from the columns an expert would have if the
// experts were chosen evenly, and the down product gives a wavefront whole experts (or a part of K by
// the number that could be used at most). Where the tokens agree on few experts both are off: 64
// tokens of one slot all to one of 64 experts (F = 1024) take 34.8 us gated and 40.2 down at D = 2048,
// 60.3 and 50.4 at D = 4096, against 27.5 and 18.3, 49.1 and 24.5 where they name 37 experts, most
// of the wavefronts of the down product having nothing to do.
#include <cmath>

#include "epilogue.h"
#include "mmq_device.h"
#include "moe_dot.h"
#include "moe_internal.h"
#include "moe_mfma.h"

namespace mmq {
namespace {

// Pair p of position i of an expert's list, kept inside the buffers whatever the plan holds.
__device__ __forceinline__ int pair_at(const int* order, int i, int P) {
  const int p = order[i];
  return p < 0 ? 0 : (p < P ? p : P - 1);
}

// p / k for a pair p (below 512) and k slots (at most 64), by the multiple m = 65535 / k + 1 of
// 2^-16: the quotient is at most 512 / 65536 = 1/128 too large, less than 1/k.
__device__ __forceinline__ int token_of(int p, int m) { return (p * m) >> 16; }

// A product's form: what its wavefronts are and how many a workgroup has.
template <class Wave, int Waves>
struct Form {
  using W = Wave;
  static constexpr int NW = Waves;
};

// ---------------------------------------------------------------- the gated product

// Workgroup (u, block): used expert u, RB blocks of W::kRows packed rows. KW wavefronts split K
// for each block (KW * RB = NW): as many as K has steps, so that a short K gives a wavefront a
// step of its own rather than none.
template <class W, int NW>
__global__ __launch_bounds__(64 * NW, 4) void moe_gated_kernel(
    const void* __restrict__ tokens, const int* __restrict__ plan,
    const uint8_t* __restrict__ wrep, float* __restrict__ H, int M, int E, int k, int F, int K,
    int entries, int act, int kw_log2, int blocks, int km) {
  constexpr int NC = W::kCols, R = W::kRows;
  __shared__ __align__(16) uint8_t smem[NW * W::kLds];
  __shared__ __align__(16) float red[NW][NC][R];
  __shared__ int pairs[NC];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int u = (int)(blockIdx.x / (unsigned)blocks), block = (int)(blockIdx.x % (unsigned)blocks);
  const int nsb = K >> 8, nsteps = (nsb + W::SB - 1) / W::SB;
  const int KW = 1 << kw_log2, RB = NW >> kw_log2;
  const int kw = wave & (KW - 1);
  const int tiles = (F + 15) >> 4;
  const int rb = block * RB + (wave >> kw_log2);
  const bool live = rb * R < 32 * tiles && kw < nsteps;
  const typename W::Tokens tk = W::tokens(tokens, M, K);
  W w;
  w.init(smem + wave * W::kLds, lds_addr(smem) + (uint32_t)(wave * W::kLds));
  typename W::Regs r;
  // one token: its values do not wait for the plan
  if constexpr (W::kFused)
    if (live) w.load_columns(tk, w.group(1, [](int) { return 0u; }), kw, nsb, 0, r);

  const int P = M * k;
  const PlanEntry en = plan_entry(plan, u, E, P);
  if (en.n == 0) return;
  const int* order = plan + kPlanHead + 4 * entries + en.first;
  const int j0 = rb * R & 31;
  const uint8_t* wtile = wrep + ((size_t)en.expert * tiles + (live ? rb * R >> 5 : 0)) *
                                    (size_t)nsb * kRepTileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wtile, (uint32_t)nsb * (uint32_t)kRepTileBytes);

  for (int g0 = 0; g0 < en.n; g0 += NC) {
    const int n = en.n - g0 < NC ? en.n - g0 : NC;
    if ((int)threadIdx.x < n) pairs[threadIdx.x] = pair_at(order, g0 + (int)threadIdx.x, P);
    const typename W::Group g = w.group(n, [&](int m) {
      return W::kFused ? 0u : (uint32_t)token_of(pair_at(order, g0 + m, P), km);
    });
    typename W::Acc acc;
    w.zero(acc);
    if (live) {
      const typename W::Src first = w.source(rw, j0, nsb, kw, true);
      w.load_weights(first, r);
      if (!W::kFused || g0 > 0) w.load_columns(tk, g, kw, nsb, 0, r);
      w.finish(tk, g, first, 0, r);
      for (int j = kw, buf = 0; j < nsteps; j += KW, buf ^= 1) {
        const bool more = j + KW < nsteps;
        const typename W::Src next = w.source(rw, j0, nsb, j + KW, more);
        w.compute(g, nsb, j, buf, r, acc, more, next, tk, g);
        if (more) w.finish(tk, g, next, buf ^ 1, r);
      }
    }
    w.each(g, acc, [&](int m, int r, auto v) {
      *reinterpret_cast<decltype(v)*>(&red[wave][m][r]) = v;
    });
    __syncthreads();
    for (int e = threadIdx.x; e < RB * NC * (R / 2); e += 64 * NW) {
      const int fl = e % (R / 2), m = e / (R / 2) % NC, bl = e / (R / 2) / NC;
      const int f = (block * RB + bl) * (R / 2) + fl, gr = 16 * (fl >> 3) + (fl & 7);
      if (m < g.n && f < F) {
        float gs = 0.0f, us = 0.0f;
        for (int i = 0; i < KW; ++i) {
          gs += red[bl * KW + i][m][gr];
          us += red[bl * KW + i][m][gr + 8];
        }
        H[(size_t)pairs[m] * F + f] = activate(gs, act) * us;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the down product

// Workgroup: W::kRows rows of the output, every used expert. A wavefront takes whole experts (or,
// where there are more wavefronts than experts, one of `wpe` parts of an expert's K), so the
// product of a pair is finished in one wavefront's registers and goes to LDS once; at the end each
// output adds its token's slots, in slot order, from there. So the sum over the slots needs no
// memory, no atomics and no second launch. The plan is copied to LDS first.
// LDS: [NW] staging, entries, y [part][position][R] of wpe * P positions, the pairs by position, the
// positions by pair, the weights.
template <class W, int NW>
__global__ __launch_bounds__(64 * NW, 4) void moe_down_kernel(
    const void* __restrict__ tokens, const int* __restrict__ plan,
    const float* __restrict__ weights, const uint8_t* __restrict__ wrep, const float* residual,
    float* out, int M, int E, int k, int N, int K, int entries, int wpe) {
  constexpr int NC = W::kCols, R = W::kRows;
  extern __shared__ __align__(16) uint8_t smem[];
  const int P = M * k;
  int4* ent = reinterpret_cast<int4*>(smem + NW * W::kLds);
  float* y = reinterpret_cast<float*>(ent + entries);
  int* ord = reinterpret_cast<int*>(y + (size_t)wpe * P * R);
  int* pos = ord + P;
  float* wts = reinterpret_cast<float*>(pos + P);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  int used = plan[0];
  if (used < 0 || used > entries) used = 0;
  for (int i = threadIdx.x; i < entries; i += 64 * NW) {
    const PlanEntry e = plan_entry(plan, i, E, P);
    ent[i] = make_int4(e.expert, e.first, e.n, 0);
  }
  const int* order = plan + kPlanHead + 4 * entries;
  for (int i = threadIdx.x; i < P; i += 64 * NW) {
    const int p = order[i];
    ord[i] = p < 0 || p >= P ? 0 : p;
    pos[i] = -1;
    wts[i] = weights[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < P; i += 64 * NW) {  // read after the barrier behind the products
    const int p = order[i];
    if (p >= 0 && p < P) pos[p] = i;
  }

  const int nsb = K >> 8, nsteps = (nsb + W::SB - 1) / W::SB;
  const int part = wave & (wpe - 1), stride = NW / wpe;
  const int rb = (int)blockIdx.x;
  const int tiles = (N + 31) >> 5;
  const int tile = rb * R >> 5, j0 = rb * R & 31;
  // the residual of this work-item's first output, read while the products run
  float res = 0.0f;
  {
    const int t = (int)threadIdx.x / R, n = rb * R + (int)threadIdx.x % R;
    if (residual && t < M && n < N) res = residual[(size_t)t * N + n];
  }
  const typename W::Tokens tk = W::tokens(tokens, P, K);
  W w;
  w.init(smem + wave * W::kLds, lds_addr(smem) + (uint32_t)(wave * W::kLds));

  // a wavefront's steps in order: its experts, their columns NC at a time, its part's steps
  struct Job {
    int u, g0, j;          // j < 0: none left
    int first, n;          // the expert's list
    const uint8_t* base;
    typename W::Group g;
  };
  // from `b` (its u, g0, j) on, the first step that there is
  auto settle = [&](Job& b) {
    if (b.g0 >= b.n) {  // another expert's first columns
      b.g0 = 0;
      b.n = 0;
      while (b.u < used) {
        const int4 e = ent[b.u];
        b.n = __builtin_amdgcn_readfirstlane(e.z);
        b.first = __builtin_amdgcn_readfirstlane(e.y);
        b.base = wrep + ((size_t)__builtin_amdgcn_readfirstlane(e.x) * tiles + tile) *
                            (size_t)nsb * kRepTileBytes;
        if (b.n) break;
        b.u += stride;
      }
    }
    b.j = b.n ? part : -1;
    if (b.n) {
      const int at = b.first + b.g0;
      b.g = w.group(b.n - b.g0 < NC ? b.n - b.g0 : NC,
                    [&](int m) { return (uint32_t)ord[at + m]; });
    }
  };
  auto advance = [&](Job& b) {
    b.j += wpe;
    if (b.j >= nsteps) {
      b.g0 += NC;
      if (b.g0 >= b.n) b.u += stride;
      settle(b);
    }
  };
  auto source = [&](const Job& b) {
    return w.source(make_rsrc(b.base, (uint32_t)nsb * (uint32_t)kRepTileBytes), j0, nsb, b.j,
                    b.j >= 0);
  };
  typename W::Acc acc;
  w.zero(acc);
  Job a;
  a.u = wave / wpe;
  a.g0 = a.first = a.n = a.j = 0;
  a.base = wrep;
  a.g = w.group(1, [](int) { return 0u; });
  settle(a);
  typename W::Regs r;
  if (a.j >= 0) {
    const typename W::Src first = source(a);
    w.load_weights(first, r);
    w.load_columns(tk, a.g, a.j, nsb, 0, r);
    w.finish(tk, a.g, first, 0, r);
  }
  for (int buf = 0; a.j >= 0; buf ^= 1) {
    Job b = a;
    advance(b);
    const typename W::Src next = source(b);
    w.compute(a.g, nsb, a.j, buf, r, acc, b.j >= 0, next, tk, b.g);
    if (b.j < 0 || b.u != a.u || b.g0 != a.g0) {
      float* to = y + ((size_t)part * P + a.first + a.g0) * R;
      w.each(a.g, acc, [&](int m, int r, auto v) {
        *reinterpret_cast<decltype(v)*>(to + m * R + r) = v;
      });
      w.zero(acc);
    }
    if (b.j >= 0) w.finish(tk, b.g, next, buf ^ 1, r);
    a = b;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < M * R; e += 64 * NW) {
    const int t = e / R, r = e % R, n = rb * R + r;
    if (n < N) {
      float v = 0.0f;
      for (int s = 0; s < k; ++s) {
        const int i = pos[t * k + s];
        if (i >= 0) {
          float d = y[(size_t)i * R + r];
          for (int q = 1; q < wpe; ++q) d += y[((size_t)q * P + i) * R + r];
          v = __builtin_fmaf(wts[t * k + s], d, v);
        }
      }
      const size_t at = (size_t)t * N + n;
      if (residual) v += e == (int)threadIdx.x ? res : residual[at];
      out[at] = v;
    }
  }
}

template <class W, int NW>
hipError_t launch_gated(const void* tokens, const int* plan, const void* w, float* H,
                        const MoeShape& m, int act, hipStream_t s) {
  const int64_t nsteps = (m.D / 256 + W::SB - 1) / W::SB;
  int kw = 0;
  while ((2 << kw) <= NW && (1 << kw) < nsteps) ++kw;
  const int64_t rb = NW >> kw, rows = 32 * ((m.F + 15) / 16);
  const int64_t blocks = (rows / W::kRows + rb - 1) / rb;
  hipLaunchKernelGGL((moe_gated_kernel<W, NW>), dim3((unsigned)(m.entries() * blocks)),
                     dim3(64 * NW), 0, s, tokens, plan, static_cast<const uint8_t*>(w), H,
                     (int)m.M, (int)m.E, (int)m.k, (int)m.F, (int)m.D, (int)m.entries(), act, kw,
                     (int)blocks, (int)(65535 / m.k + 1));
  return hipGetLastError();
}

// Parts of an expert's K in the down product: as many as there are wavefronts per entry, steps,
// and room for (512 positions of y, or the pairs).
template <class W, int NW>
int64_t down_parts(const MoeShape& m) {
  const int64_t nsteps = (m.F / 256 + W::SB - 1) / W::SB;
  int64_t wpe = 1;
  while (2 * wpe * m.entries() <= NW && 2 * wpe <= nsteps && 2 * wpe * m.pairs() <= 512) wpe *= 2;
  return wpe;
}

template <class W, int NW>
int64_t down_lds(const MoeShape& m) {
  return NW * W::kLds + 16 * m.entries() + 12 * m.pairs() +
         4 * down_parts<W, NW>(m) * m.pairs() * W::kRows;
}

template <class W, int NW>
hipError_t launch_down(const void* tokens, const int* plan, const float* weights, const void* w,
                       const float* residual, float* out, const MoeShape& m, hipStream_t s) {
  auto kern = moe_down_kernel<W, NW>;
  const int64_t lds = down_lds<W, NW>(m);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)((m.D + W::kRows - 1) / W::kRows)), dim3(64 * NW),
                     (size_t)lds, s, tokens, plan, weights, static_cast<const uint8_t*>(w),
                     residual, out, (int)m.M, (int)m.E, (int)m.k, (int)m.D, (int)m.F,
                     (int)m.entries(), (int)down_parts<W, NW>(m));
  return hipGetLastError();
}

// Columns per used expert, were the experts chosen evenly: the M * k pairs over the
// E (1 - (1 - k/E)^M) experts that some token names.
double columns_per_expert(const MoeShape& m) {
  const double used = (double)m.E * (1.0 - std::pow(1.0 - (double)m.k / (double)m.E, (double)m.M));
  return (double)m.pairs() / used;
}

// f of a down product's form.
template <class F>
auto with_down(const MoeShape& m, int64_t compute_units, F f) {
  // 8 rows per workgroup while those workgroups run in one round (an output of few rows would
  // leave compute units idle with 16), else 16. One token, graph replays over weights beyond the
  // cache, 8 of 64 experts of F = 1024: 8 rows 7.8, 16 rows 8.1 us at D = 2048, but 12.6 against
  // 8.0 us at 2560.
  const bool narrow = (m.D + 7) / 8 <= compute_units;
  if (moe_fused(m.M))
    return narrow ? f(Form<DotWave<8, 1, true>, 16>{})
                  : f(Form<DotWave<16, 1, true>, 16>{});
  const double c = columns_per_expert(m);
  // The vector-ALU form for few columns (graph replays over weights beyond the cache, vector ALU
  // against matrix unit). D = 2048: at 1.2 columns (4 tokens, 8 of 64 experts of F = 1024) 13.2
  // against 14.7 us, at 1.5 (8 tokens) 16.8 against 19.3, at 2.4 (23 tokens, 6 of 64, F = 1280) 30.9
  // against 30.6 (29.5 against 24.9 while the weights fit the cache), at 8 (64 tokens) 52.7 against
  // 44.0. D = 4096: at 1.5 (4 tokens, 2 of 8, F = 11008) 33.8 against 47.4, at 3.1 (12 tokens, 4 of
  // 16, F = 4096) 40.3 against 41.9, at 4 (16 tokens, 2 of 8) 57.9 against 58.2, but 58.2 against 43.1
  // for 16 tokens, 4 of 16, whose most liked expert has 13 columns, four groups of 4; at 16 (64 tokens)
  // 183 against 103. Its step is twice the matrix unit's bytes per wavefront, which counts while
  // loads in flight set the rate.
  if (narrow)
    return c <= 2.0 ? f(Form<DotWave<8, 3, false>, 16>{})
                    : f(Form<MfmaWave<1, 2>, 16>{});
  return c <= 5.0 ? f(Form<DotWave<16, 4, false>, 16>{})
                  : f(Form<MfmaWave<1>, 16>{});
}

}  // namespace

hipError_t launch_moe_gated(const void* tokens, const int* plan, const void* w, float* H,
                            const MoeShape& m, int act, hipStream_t s) {
  // One token: the vector ALU, from float32, one launch. Else the matrix unit: with one or two
  // columns it takes what the vector-ALU form with up to 4 took (graph replays: 2 tokens, 2 of 8
  // experts, D = 4096, F = 11008, 46 us both; 4 tokens 66.3 against 66.9), with 4 columns 95 against
  // 107, and with 16 (64 tokens) 139 against 278. Two wavefronts per workgroup, so that each walks
  // half of K: the prologue and the sum over wavefronts weigh less (4 and 8 tokens were slower by
  // up to 8 %), while one per workgroup leaves the short K of small experts unsplit.
  if (moe_fused(m.M)) return launch_gated<DotWave<16, 1, true>, 4>(tokens, plan, w, H, m, act, s);
  // Above 8 columns on average some experts have more than 16: their weights are read again. Loaded as
  // read once against not, D = 4096: 8 columns (64 tokens, 8 of 64, F = 1024) 82.2 / 85.8 us, 9 (36
  // tokens, 2 of 8, F = 11008) 108.2 / 110.7, 12 (48) 112.8 / 114.7, 16 (64) 149.7 / 142.4: the two
  // sides meet between 12 and 16, and the switch at 8 costs 2 % between.
  return columns_per_expert(m) <= 8.0
             ? launch_gated<MfmaWave<2, 1, true>, 2>(tokens, plan, w, H, m, act, s)
             : launch_gated<MfmaWave<2>, 2>(tokens, plan, w, H, m, act, s);
}

hipError_t launch_moe_down(const void* tokens, const int* plan, const float* weights,
                           const void* w, const float* residual, float* out, const MoeShape& m,
                           int64_t compute_units, hipStream_t s) {
  return with_down(m, compute_units, [&](auto form) {
    using T = decltype(form);
    return launch_down<typename T::W, T::NW>(tokens, plan, weights, w, residual, out, m, s);
  });
}

int64_t moe_down_lds_bytes(const MoeShape& m, int64_t compute_units) {
  return with_down(m, compute_units, [&](auto form) {
    using T = decltype(form);
    return down_lds<typename T::W, T::NW>(m);
  });
}

}  // namespace mmq
