// The (token, slot) pairs sorted by expert, for the products grouped by expert, and the weighted sum
// over a token's slots behind them.
//
// The sort is a counting sort that keeps the order of equal keys: the place of pair p is
//   offsets[e] + #{p' < p : expert(p') = e},  offsets[e] = #{p : expert(p) < e},
// so there is one result and it does not depend on any order of execution. A wavefront takes 64
// consecutive pairs at a time: the lanes with the same expert are found by one ballot per bit of the
// expert's number, a lane's rank is the number of such lanes below it, and the lowest of them adds
// their count to the wavefront's own row of counts in LDS. The rows of the 16 wavefronts are then
// added up expert by expert. Nothing is added atomically.
//
// Bound by latency: reads of the ids, LDS round trips and launches. Up to 4096 pairs one workgroup does it
// (graph replays, a launch being 3.6 us: 800 pairs 3.7 us, 2000 4.7, 4096 6.5); above, chunks of 2048 pairs in
// two kernels (4100 pairs 7.6 us, 16384 8.1, 65536 of 256 experts 9.3, 2^21 86, 2^21 of 512 experts 153: every
// workgroup of the second reads the counts of all chunks), which take as long as that for fewer pairs too.
// Chunks of 4096 with the counts added up by one work-item per expert and the ranks found twice took 12.4 us for
// the 65536.
#include "grouped_internal.h"

namespace mmq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

struct SortLds {
  int count[kWaves][kGroupMaxExperts];
  int base[kGroupMaxExperts];
  int wave_total[kWaves];
};

// The lanes of the wavefront whose key equals this lane's; keys are below 2^bits.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t with = __ballot(one);
    m &= one ? with : ~with;
  }
  return m;
}

// Ranks within the workgroup's NI * 1024 pairs from p0 on: id[i] the expert of this thread's i-th
// pair (E where it has none), rank[i] how many pairs of that expert its wavefront saw before;
// sh.count[w][e] becomes how many the wavefronts below w saw, and total the workgroup's count of
// expert threadIdx.x.
template <int NI>
__device__ __forceinline__ void rank_pairs(SortLds& sh, const int* __restrict__ ids, int64_t p0,
                                           int64_t P, int E, int bits, int (&id)[NI],
                                           int (&rank)[NI], int& total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = p0 + (int64_t)wave * (64 * NI) + lane;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t p = first + 64 * i;
    const int v = p < P ? ids[p] : -1;
    id[i] = v >= 0 && v < E ? v : E;
  }
  for (int e = tid; e < kWaves * kGroupMaxExperts; e += kThreads) (&sh.count[0][0])[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint64_t m = same_key(id[i], bits);
    const int below = __popcll(m & ((1ull << lane) - 1ull));
    int before = 0;
    if (id[i] < E) before = sh.count[wave][id[i]];
    rank[i] = before + below;
    // the wavefront's reads above come before this write: one wavefront's LDS operations are in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (id[i] < E && below == 0) sh.count[wave][id[i]] = before + __popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  total = 0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = sh.count[w][tid];
      sh.count[w][tid] = total;
      total += n;
    }
  }
}

// sh.base[e] = the sum of n over the experts below e; returns the sum over all of them.
__device__ __forceinline__ int scan_experts(SortLds& sh, int n, int E) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int incl = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) sh.wave_total[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWaves; ++w) {
    const int v = sh.wave_total[w];
    if (w < wave) before += v;
    all += v;
  }
  if (tid < E) sh.base[tid] = before + incl - n;
  __syncthreads();
  return all;
}

template <int NI>
__device__ __forceinline__ void write_places(const SortLds& sh, int64_t P, int E,
                                             int all, const int (&id)[NI], const int (&rank)[NI],
                                             int* __restrict__ order, int* __restrict__ place) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)wave * (64 * NI) + lane;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t p = first + 64 * i;
    if (p >= P) continue;
    int at = -1;
    if (id[i] < E) {
      at = sh.base[id[i]] + sh.count[wave][id[i]] + rank[i];
      order[at] = (int)p;
    }
    place[p] = at;
    if (p >= all) order[p] = -1;
  }
}

// All pairs in one workgroup.
template <int NI>
__global__ __launch_bounds__(kThreads) void group_kernel(const int* __restrict__ ids, int P, int E,
                                                         int bits, int* __restrict__ groups) {
  __shared__ SortLds sh;
  int id[NI], rank[NI], total;
  rank_pairs<NI>(sh, ids, 0, P, E, bits, id, rank, total);
  const int all = scan_experts(sh, total, E);
  const GroupLayout g{P, E};
  if ((int)threadIdx.x < E) groups[threadIdx.x] = sh.base[threadIdx.x];
  if (threadIdx.x == 0) groups[E] = all;
  write_places<NI>(sh, P, E, all, id, rank, groups + g.order(), groups + g.place());
}

// Many pairs, in chunks of kGroupChunk: the counts of each chunk, and in `place` the rank of each pair in
// its chunk ...
constexpr int kChunkNI = kGroupChunk / kThreads;
__global__ __launch_bounds__(kThreads) void count_kernel(const int* __restrict__ ids, int64_t P,
                                                         int E, int bits, int* __restrict__ groups) {
  __shared__ SortLds sh;
  const GroupLayout g{P, E};
  const int64_t p0 = (int64_t)blockIdx.x * kGroupChunk;
  int id[kChunkNI], rank[kChunkNI], total;
  rank_pairs<kChunkNI>(sh, ids, p0, P, E, bits, id, rank, total);
  if ((int)threadIdx.x < E)
    groups[g.counts() + (int64_t)blockIdx.x * E + threadIdx.x] = total;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < kChunkNI; ++i) {
    const int64_t p = p0 + (int64_t)wave * (64 * kChunkNI) + 64 * i + lane;
    if (p < P && id[i] < E) groups[g.place() + p] = sh.count[wave][id[i]] + rank[i];
  }
}

// ... and, with the counts of the chunks before it, the places. The counts are read by all work-items, one
// to an expert and a share of the chunks.
__global__ __launch_bounds__(kThreads) void place_kernel(const int* __restrict__ ids, int64_t P,
                                                         int E, int* __restrict__ groups) {
  __shared__ SortLds sh;
  const GroupLayout g{P, E};
  const int64_t p0 = (int64_t)blockIdx.x * kGroupChunk;
  const int tid = threadIdx.x;
  int* order = groups + g.order();
  int* place = groups + g.place();
  int id[kChunkNI], rank[kChunkNI];
#pragma unroll
  for (int i = 0; i < kChunkNI; ++i) {
    const int64_t p = p0 + i * kThreads + tid;
    const int v = p < P ? ids[p] : -1;
    id[i] = v >= 0 && v < E ? v : E;
    rank[i] = id[i] < E ? place[p] : 0;
  }
  int wide = 64;  // experts, rounded up to a power of two
  while (wide < E) wide *= 2;
  const int e = tid & (wide - 1), share = tid / wide, shares = kThreads / wide;
  int n = 0, before = 0;
  if (e < E) {
    const int* c = groups + g.counts() + e;
    const int chunks = (int)g.chunks();
#pragma unroll 8
    for (int i = share; i < chunks; i += shares) {
      const int v = c[(int64_t)i * E];
      n += v;
      if (i < (int)blockIdx.x) before += v;
    }
  }
  // shares of an expert in sh.count, as [share][n, before][expert]
  int* part = &sh.count[0][0];
  static_assert(2 * kThreads <= kWaves * kGroupMaxExperts, "LDS of the shares");
  part[2 * share * wide + e] = n;
  part[(2 * share + 1) * wide + e] = before;
  __syncthreads();
  n = before = 0;
  if (tid < E)
    for (int i = 0; i < shares; ++i) {
      n += part[2 * i * wide + tid];
      before += part[(2 * i + 1) * wide + tid];
    }
  const int all = scan_experts(sh, n, E);
  if (blockIdx.x == 0) {
    if (tid < E) groups[tid] = sh.base[tid];
    if (tid == 0) groups[E] = all;
  }
  if (tid < E) sh.base[tid] += before;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kChunkNI; ++i) {
    const int64_t p = p0 + i * kThreads + tid;
    if (p >= P) continue;
    int at = -1;
    if (id[i] < E) {
      at = sh.base[id[i]] + rank[i];
      order[at] = (int)p;
    }
    place[p] = at;
    if (p >= all) order[p] = -1;
  }
}

// One work-item per four (or one) columns of a token.
template <bool VEC4>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ Y,
                                                      const int* __restrict__ place,
                                                      const float* __restrict__ weights,
                                                      const float* residual, float* out, int64_t M,
                                                      int k, int64_t D) {
  const int64_t per = VEC4 ? D / 4 : D;
  const int64_t groups = (per + 255) / 256;
  const int64_t t = (int64_t)blockIdx.x / groups;
  const int64_t c = ((int64_t)blockIdx.x - t * groups) * 256 + threadIdx.x;
  if (c >= per) return;
  const int* pl = place + t * k;
  const float* w = weights + t * k;
  const float* y = Y + t * k * D;
  if constexpr (VEC4) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t at = t * D + 4 * c;
    if (residual) a = *reinterpret_cast<const float4*>(residual + at);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < k; ++s) {
      if (pl[s] < 0) continue;
      const float4 v = *reinterpret_cast<const float4*>(y + s * D + 4 * c);
      sum.x = __builtin_fmaf(w[s], v.x, sum.x);
      sum.y = __builtin_fmaf(w[s], v.y, sum.y);
      sum.z = __builtin_fmaf(w[s], v.z, sum.z);
      sum.w = __builtin_fmaf(w[s], v.w, sum.w);
    }
    *reinterpret_cast<float4*>(out + at) =
        make_float4(sum.x + a.x, sum.y + a.y, sum.z + a.z, sum.w + a.w);
  } else {
    const int64_t at = t * D + c;
    float sum = 0.0f;
    for (int s = 0; s < k; ++s)
      if (pl[s] >= 0) sum = __builtin_fmaf(w[s], y[s * D + c], sum);
    out[at] = residual ? sum + residual[at] : sum;
  }
}

}  // namespace

hipError_t launch_group(const int* ids, int64_t P, int64_t E, int* groups, hipStream_t s) {
  int bits = 1;
  while (((int64_t)1 << bits) <= E) ++bits;  // the key E is a pair without an expert
  const int p = (int)P, e = (int)E;
  if (P <= kThreads) {
    hipLaunchKernelGGL(group_kernel<1>, dim3(1), dim3(kThreads), 0, s, ids, p, e, bits, groups);
  } else if (P <= 2 * kThreads) {
    hipLaunchKernelGGL(group_kernel<2>, dim3(1), dim3(kThreads), 0, s, ids, p, e, bits, groups);
  } else if (P <= kGroupOne) {
    hipLaunchKernelGGL(group_kernel<4>, dim3(1), dim3(kThreads), 0, s, ids, p, e, bits, groups);
  } else {
    const dim3 grid((unsigned)GroupLayout{P, E}.chunks());
    hipLaunchKernelGGL(count_kernel, grid, dim3(kThreads), 0, s, ids, P, e, bits, groups);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(place_kernel, grid, dim3(kThreads), 0, s, ids, P, e, groups);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const float* Y, const int* place, const float* weights,
                          const float* residual, float* out, int64_t M, int64_t k, int64_t D,
                          hipStream_t s) {
  const bool vec = D % 4 == 0;
  const int64_t per = vec ? D / 4 : D;
  const dim3 grid((unsigned)((per + 255) / 256 * M));
  if (vec)
    hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, s, Y, place, weights, residual, out,
                       M, (int)k, D);
  else
    hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, s, Y, place, weights, residual,
                       out, M, (int)k, D);
  return hipGetLastError();
}

}  // namespace mmq
