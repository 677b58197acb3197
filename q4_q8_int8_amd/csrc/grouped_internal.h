// The products grouped by expert: shared declarations (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mmq_internal.h"

namespace mmq {

constexpr int64_t kGroupMaxPairs = (int64_t)1 << 21;
constexpr int kGroupMaxExperts = 512;

// The groups of P = M*k pairs over E experts, int32, each part at a multiple of four words:
// offsets[E + 1], order[P], place[P], then the sort's own counts (chunks of pairs by experts).
// The sort: pairs of one workgroup that does it alone, and of one of several.
constexpr int kGroupOne = 4096, kGroupChunk = 2048;
__host__ __device__ constexpr int64_t round4(int64_t v) { return (v + 3) / 4 * 4; }
struct GroupLayout {
  int64_t P, E;
  __host__ __device__ constexpr int64_t order() const { return round4(E + 1); }
  __host__ __device__ constexpr int64_t place() const { return order() + round4(P); }
  __host__ __device__ constexpr int64_t counts() const { return place() + round4(P); }
  __host__ __device__ constexpr int64_t chunks() const {
    return (P + kGroupChunk - 1) / kGroupChunk;
  }
  __host__ __device__ constexpr int64_t words() const {
    return counts() + (P > kGroupOne ? round4(chunks() * E) : 0);
  }
};

hipError_t launch_group(const int* ids, int64_t P, int64_t E, int* groups, hipStream_t s);

// A product over the groups: N weight rows (kEpiGated: packed rows) of E matrices, K values each.
// Row p of the output is pair p's; its activations are row p / per_row of the q8 buffer (of q_rows
// rows): per_row = k for one row per token, 1 for one per pair.
struct GroupedShape {
  int64_t P, E, N, K, q_rows, per_row;
};
// The kernel's form for a shape, chosen by a cost model (grouped.hip) as if the pairs fell evenly on
// the experts, and its LDS.
enum GroupedForm { kGroupedWide, kGroupedNarrow, kGroupedSplit2, kGroupedSplit4 };
GroupedForm grouped_form(const GroupedShape& g, int64_t compute_units);
int64_t grouped_lds_bytes(GroupedForm f);
// The q8 buffer is quantize_q8_1's but for its float pairs, which are [M][K/32] here (row by row,
// so that the rows of a group can be gathered); K % 256 == 0.
hipError_t launch_quantize_rows(const float* x, int64_t M, int64_t K, void* q8, hipStream_t s);
hipError_t launch_grouped(const void* q8, const int* groups, const void* w, float* out,
                          const GroupedShape& g, const Epilogue& epi, int64_t compute_units,
                          hipStream_t s);

// out[t][D] = residual[t] + sum over s of weights[t][s] * Y[t*k + s], over the pairs with an expert.
hipError_t launch_combine(const float* Y, const int* place, const float* weights,
                          const float* residual, float* out, int64_t M, int64_t k, int64_t D,
                          hipStream_t s);

}  // namespace mmq
