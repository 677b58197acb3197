// Matrix-vector products with 4-bit weights and group scales: shared declarations (not part of the
// ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mmq_internal.h"

namespace mmq {

// enum mmq_type, restated for the kernels
constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBF16 = 2;

// Repacked weights: first the values, one 1024-byte record per (tile of 16 rows, 128 values),
// [tile][record]; then at a 256-byte boundary the scales, 16-bit [tile][group][16 rows]; then, the
// same way, the zeros. Rows past N and values past K are 0. A record holds dwords
// [c 0..3][row 0..15][m 0..3] of the 8 values k = 128 record + 32 m + 8 c + e of a row: value e = 2 j
// in nibble j, e = 2 j + 1 in nibble j + 4, so that one 16-byte load per lane gives the rows of four
// 16 x 16 x 32 matrix instructions, and an AND and a shift by at most 12 bits the two halves of each
// operand register.
constexpr int kG4Rows = 16, kG4Values = 128, kG4RecBytes = 1024;
constexpr int kG4MaxTokens = 16;

struct Q4GShape {
  int64_t N, K, group;
  bool zeros;
  constexpr int64_t tiles() const { return (N + kG4Rows - 1) / kG4Rows; }
  constexpr int64_t records() const { return (K + kG4Values - 1) / kG4Values; }
  constexpr int64_t groups() const { return (K + group - 1) / group; }
  constexpr int64_t scales_at() const { return tiles() * records() * kG4RecBytes; }
  constexpr int64_t zeros_at() const { return round256(scales_at() + tiles() * groups() * 32); }
  constexpr int64_t bytes() const {
    return zeros ? zeros_at() + tiles() * groups() * 32 : scales_at() + tiles() * groups() * 32;
  }
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
