// Products of 8-bit floating-point operands with a scale for every 128 entries
// of the inner dimension:
//   C(i, j) = sum over blocks b of SA(i, b) SB(j, b) (sum over k in b of A(k, i) B(k, j))
// Declarations for the kernels (gemm8.hip) and their host side (scaled.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ozgemm.h"

namespace oz {

// Rows of q bytes, K-contiguous, beginning on 16-byte boundaries.
struct Operand8 {
  const uint8_t* p;
  long ld;
  const float* s;
  long srow, sblock;  // scale of row i and block b: s[(i >> shift) srow + b sblock]
  int shift;          // 0: every row its own; 7: 128 rows share one
};

struct Scaled8 {
  Operand8 A, B;  // B's shift is 0
  int atype, btype;
  int m, n, q;  // A's rows, B's rows, inner dimension
  void* C;
  int ctype;
  long ldc;
  int parts;       // of the inner dimension
  float* partial;  // their sums, [parts][n][m]
};

// Largest leading dimension: 256 rows of it stay within 32-bit offsets.
constexpr long LD8_MAX = 1L << 22;

// Parts of the inner dimension a product of these sizes is summed in.
int scaled_parts(int m, int n, int q);
// Whether the launches have at most 2^32 - 1 threads each.
bool scaled_fits(int m, int n, int parts);
hipError_t launch_scaled(const Scaled8& g, hipStream_t st);

// Whether a product of these sizes goes by the largest tiles.
bool scaled_big(int m, int n, int q);

// the scales (row, block) of rows of q entries to block rows + row
hipError_t launch_turn_scales(const float* src, long srow, long sblock, int rows, int q, float* dst, hipStream_t st);

// rows x q bytes, rows ld apart, to rows up(q, 16) apart
hipError_t launch_align_rows(const uint8_t* src, long ld, int rows, int q, uint8_t* dst, long dld, hipStream_t st);

}  // namespace oz
