// Matrix-vector products with 4-bit weights and group scales: shared declarations (not part of the
// ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mmq_internal.h"

namespace mmq {

// enum mmq_type, restated for the kernels
constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBF16 = 2;

// Repacked weights: one record per (tile of 16 rows, 128 values), [tile][record], rows past N and
// values past K being 0. A record holds
//   1024 bytes  dwords [c 0..3][row 0..15][m 0..3] of the 8 values k = 128 record + 32 m + 8 c + e of a
//               row: value e = 2 j in nibble j, e = 2 j + 1 in nibble j + 4. One 16-byte load per lane is
//               what four 16 x 16 x 32 matrix instructions take, and a shift and an AND make two values
//               of a dword an operand register.
//   32 S bytes  16-bit scales [row][S], and, where there are zeros, as many bytes of those. S is how
//               many scales a row has in a record: 1 where its 128 values lie in one group, 2 for groups
//               of 64, else 4, one per 32 values.
constexpr int kG4Rows = 16, kG4Values = 128, kG4ValueBytes = 1024;
constexpr int kG4MaxTokens = 16;

struct Q4GShape {
  int64_t N, K, group;
  bool zeros;
  constexpr int64_t tiles() const { return (N + kG4Rows - 1) / kG4Rows; }
  constexpr int64_t records() const { return (K + kG4Values - 1) / kG4Values; }
  constexpr int64_t groups() const { return (K + group - 1) / group; }
  constexpr int scales() const {
    return group % kG4Values == 0 || group >= K ? 1 : group == kG4Values / 2 ? 2 : 4;
  }
  constexpr int64_t record_bytes() const {
    return kG4ValueBytes + 2 * kG4Rows * scales() * (zeros ? 2 : 1);
  }
  constexpr int64_t bytes() const { return tiles() * records() * record_bytes(); }
};

struct Q4GEpilogue {
  const float* bias;     // [N] or null
  const void* residual;  // [M][N] of the output's type, or null; may be the output
  int act;
};

hipError_t launch_repack_q4g(const void* w, const void* scales, const void* zeros,
                             const Q4GShape& g, void* rep, hipStream_t s);
// M <= kG4MaxTokens tokens of x_type, results of y_type, scales of scale_type.
hipError_t launch_q4g(const void* x, int x_type, const void* rep, int scale_type, void* y,
                      int y_type, int64_t M, const Q4GShape& g, const Q4GEpilogue& epi,
                      int64_t compute_units, hipStream_t s);
int64_t q4g_lds_bytes(int x_type, int64_t M, const Q4GShape& g, int64_t compute_units);

}  // namespace mmq
