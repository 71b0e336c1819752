// Internal declarations of the grouped products and the orthogonalisation.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ozgemm.h"

namespace oz {

inline size_t elem_bytes(int type) {
  return type == OZGEMM_F64 ? 8 : type == OZGEMM_F32 ? 4 : 2;
}

inline size_t up(size_t x, size_t r) { return (x + r - 1) / r * r; }

// An operand of a 16-bit product as the kernels read it.
struct Operand16 {
  const uint16_t* p;
  long ld;     // elements between rows (K-contiguous) or between k (K-strided)
  long batch;  // elements between the matrices of two groups (0: one matrix for all)
  long plane;  // elements between the two slices (0: one slice)
  bool ks;     // K-strided
  long last;   // entries that may be read of the last row (K-strided: of the last k)
  const int32_t* ex;  // exponents of the rows (nullptr: none), ex_batch apart between groups
  long ex_batch;
};

struct Grouped16 {
  Operand16 A, B;
  int bf16;   // the slices' type: 1 bfloat16, 0 half
  int f32;    // two half slices each (few columns: as they are)
  bool few;   // by the kernels for few columns or small outer products
  bool edge;  // which then must not take runs of 16 bytes for aligned or whole
  int m, n, q, groups;
  const int32_t* offsets;
  void* C;
  int ctype;
  long ldc, cbatch;
  int parts;       // of the inner dimension (outer products: of each group's columns)
  int units, skip;  // compute units; blocks left out of the launch (share.h)
  float* partial;  // their sums: [parts][n][m] (outer products: [parts][groups][q][m])
};

// Whether the launches below have at most 2^31 - 1 tiles.
bool grouped_n_fits(const Grouped16& g);
bool grouped_k_fits(const Grouped16& g);
// C(:, J_e) = A_e B(:, J_e): B's rows are the n columns of the call.
hipError_t launch_grouped_n(const Grouped16& g, hipStream_t st);
// Whether a product of these sizes goes by the kernels for few columns: 0, or
// the parts of its inner dimension.  They read any operands as they lie; the
// others need slices of F32 and copies of those off the 16-byte grid (`edge`).
int few_columns_parts(bool f32, bool edge, bool a_strided, int groups, int m, int n, int q);
// Parts for a product of these sizes, and the room they take: where its tiles
// are too few for the card and its inner dimension is long.
int gemm_parts(bool f32, int groups, int m, int n, int q);
size_t gemm_partial_bytes(int parts, int m, int n);
int outer_parts(bool f32, int groups, int m, int q, int n);
size_t outer_partial_bytes(int parts, int groups, int m, int q);
// The same for the kernel for small outer products.
int few_outer_parts(bool f32, bool edge, int groups, int m, int q, int n);
// C_e (m x q) = sum over j in J_e: A's and B's inner dimension is the n columns.
hipError_t launch_grouped_k(const Grouped16& g, hipStream_t st);

// slices.hip ---------------------------------------------------------------
// Operands laid out for the 16-bit products: K-contiguous planes whose rows
// are padded with zeros to a multiple of 64.

// rows x K, element (r, k) at src[r ld + k]; `batches` of them, `sbatch` apart
hipError_t launch_slice_rows(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st);
// element (r, k) at src[k ld + r], `batches` of them, `sbatch` apart; part:
// slice_part_bytes of scratch (F32)
hipError_t launch_slice_cols(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, uint32_t* part, hipStream_t st);
size_t slice_part_bytes(int rows, long K, int groups, bool ragged);
// element (r, k) at src[k ld + r], k in groups that begin at offsets[e]; group
// e's rows begin at 64 x (its 64-tiles before); ex[e rows + r]
hipError_t launch_slice_groups(int type, const void* src, long ld, int rows, int n, const int32_t* offsets,
                               int groups, uint16_t* dst, long dld, long plane, int32_t* ex, uint32_t* part,
                               hipStream_t st);

// ozgemm.hip: Scheme II products in a region of a caller's workspace
// (conservative budget, no configuration; the region holds every product of
// an r x c matrix's iteration).
size_t dgemm_region_bytes(int r, int c, int s);
hipError_t dgemm_region_table(char* region, int s, hipStream_t st);  // once before the products of a call
// C (m x n) = A^T B with A q x m and B q x n, q >= 1; A may be B.
int dgemm_region_tn(char* region, int m, int n, int q, const double* A, int lda, const double* B, int ldb, double* C,
                    int ldc, int s, hipStream_t st);

// Compute units of the current device.
hipError_t device_units(int* cus);

// Keep the name of a HIP error for ozgemm_strerror and return OZGEMM_HIP_ERROR.
int record_hip_error(hipError_t err);

}  // namespace oz
