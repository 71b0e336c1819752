// Host side of the grouped products: argument checks, how each operand is
// read (in place or through slices in the workspace), and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "products.h"
#include "tile16.h"

namespace oz {
namespace {

constexpr size_t WS_ALIGN = 256;

bool known_type(int type) { return type == OZGEMM_F32 || type == OZGEMM_BF16 || type == OZGEMM_F16; }

// `run`: entries in 16 bytes
bool aligned16(const void* p, long ld, long batch, int run = 8) {
  return ((uintptr_t)p & 15) == 0 && ld % run == 0 && batch % run == 0 && ld <= LD16_MAX;
}

// Bytes from the first entry of `batches` rows x cols column-major matrices
// to the end of the last.
size_t extent(int rows, long cols, long ld, long long batch, int batches, size_t size) {
  if (rows < 1 || cols < 1 || batches < 1) return 0;
  return ((size_t)(batches - 1) * (size_t)batch + (size_t)(cols - 1) * (size_t)ld + (size_t)rows) * size;
}

bool overlap(const void* a, size_t abytes, const void* b, size_t bbytes) {
  const char* pa = (const char*)a;
  const char* pb = (const char*)b;
  return abytes && bbytes && pa < pb + bbytes && pb < pa + abytes;
}

// Room for one operand laid out in the workspace.
struct Room {
  bool used;
  long ld;        // entries per row
  size_t plane;   // entries per slice
  size_t at, ex;  // offsets of the slices and of the exponents
  size_t part;    // of the partial maxima of K-strided F32 entries
};

size_t take(size_t& total, size_t bytes) {
  const size_t at = total;
  total += up(bytes, WS_ALIGN);
  return at;
}

Room room(int type, bool used, size_t rows, size_t k, size_t exponents, size_t part, size_t& total) {
  Room r{used, (long)up(k, 64), 0, 0, 0, 0};
  if (!used) return r;
  r.plane = rows * (size_t)r.ld;
  r.at = take(total, r.plane * 2 * (type == OZGEMM_F32 ? 2 : 1));
  if (type == OZGEMM_F32) {
    r.ex = take(total, exponents * 4);
    r.part = take(total, part);
  }
  return r;
}

struct Rooms {
  Room A, B;
  int few;         // the kernels for few columns or small outer products take it (0: no)
  bool edge;       // operands off the 16-byte grid
  int parts;       // of the inner dimension
  size_t partial;  // offset of their sums
  size_t total;
};

Rooms gemm_rooms(int type, int groups, int m, int n, int q, int transa, const void* A, int lda, long long stridea,
                 const void* B, int ldb) {
  const bool f32 = type == OZGEMM_F32;
  Rooms r{};
  const int run = f32 ? 4 : 8;
  const bool a_fits = aligned16(A, lda, stridea, run) && (transa ? q : m) % run == 0;
  const bool b_fits = aligned16(B, ldb, 0, run) && q % run == 0;
  r.edge = !a_fits || !b_fits;
  if (m > 0 && n > 0 && groups > 0) r.few = few_columns_parts(f32, r.edge, transa == 0, groups, m, n, q);
  const bool a_in_place = r.few || (a_fits && !f32), b_in_place = r.few || (b_fits && !f32);
  const bool any = m > 0 && n > 0 && q > 0 && groups > 0;
  r.A = room(type, any && !a_in_place, (size_t)groups * m, q, (size_t)groups * m,
             transa ? 0 : slice_part_bytes(m, q, groups, false), r.total);
  r.B = room(type, any && !b_in_place, n, q, n, 0, r.total);
  r.parts = !any ? 1 : r.few ? r.few : gemm_parts(f32, groups, m, n, q);
  r.partial = take(r.total, gemm_partial_bytes(r.parts, m, n));
  return r;
}

Rooms outer_rooms(int type, int groups, int m, int q, int n, const void* A, int lda, const void* B, int ldb) {
  Rooms r{};
  const bool f32 = type == OZGEMM_F32;
  const int run = f32 ? 4 : 8;
  r.edge = !aligned16(A, lda, 0, run) || !aligned16(B, ldb, 0, run) || m % run != 0 || q % run != 0;
  if (m > 0 && q > 0 && groups > 0) r.few = few_outer_parts(f32, r.edge, groups, m, q, n);
  const bool in_place = r.few || (!f32 && !r.edge);
  const bool any = m > 0 && n > 0 && q > 0 && groups > 0;
  // every group's columns begin at a multiple of 64
  const size_t k = (size_t)n + 63 * (size_t)std::min(groups, n);
  r.A = room(type, any && !in_place, m, k, (size_t)groups * m, slice_part_bytes(m, n, groups, true), r.total);
  r.B = room(type, any && !in_place, q, k, (size_t)groups * q, slice_part_bytes(q, n, groups, true), r.total);
  r.parts = !any ? 1 : r.few ? r.few : outer_parts(f32, groups, m, q, n);
  r.partial = take(r.total, outer_partial_bytes(r.parts, groups, m, q));
  return r;
}

Operand16 in_place(const void* p, long ld, long batch, bool ks, int last) {
  return Operand16{(const uint16_t*)p, ld, batch, 0, ks, last, nullptr, 0};
}

Operand16 sliced(int type, const Room& r, char* ws, long batch, long ex_batch) {
  return Operand16{(const uint16_t*)(ws + r.at), r.ld, batch, (long)r.plane, false, r.ld,
                   type == OZGEMM_F32 ? (const int32_t*)(ws + r.ex) : nullptr, ex_batch};
}

#define OZ_TRY(expr)                                                   \
  do {                                                                 \
    const hipError_t oz_err_ = (expr);                                 \
    if (oz_err_ != hipSuccess) return record_hip_error(oz_err_);       \
  } while (0)

bool too_long(int m, int n, int q, int groups) {
  return m > OZGEMM_MAX_ROWS || n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS || groups > OZGEMM_GROUPS_MAX;
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozgemm_grouped_gemm_workspace_bytes(int type, int groups, int m, int n, int q, int transa, const void* A,
                                           int lda, long long stridea, const void* B, int ldb) {
  if (!known_type(type) || groups < 0 || m < 0 || n < 0 || q < 0 || too_long(m, n, q, groups)) return 0;
  return gemm_rooms(type, groups, m, n, q, transa, A, lda, stridea, B, ldb).total;
}

int ozgemm_grouped_gemm(int type, int ctype, int groups, int m, int n, int q, int transa, const void* A, int lda,
                        long long stridea, const void* B, int ldb, const int32_t* offsets, void* C, int ldc,
                        void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!known_type(type)) return -1;
  if (ctype != type && ctype != OZGEMM_F32) return -2;
  if (groups < 0) return -3;
  if (m < 0) return -4;
  if (n < 0) return -5;
  if (q < 0) return -6;
  if (transa != 0 && transa != 1) return -7;
  const bool any = m > 0 && n > 0 && groups > 0;
  const int ar = transa ? q : m, ac = transa ? m : q;
  if (A == nullptr && any && q > 0) return -8;
  if (lda < std::max(1, ar)) return -9;
  if (stridea < 0) return -10;
  if (B == nullptr && any && q > 0) return -11;
  if (ldb < std::max(1, q)) return -12;
  if (offsets == nullptr && any) return -13;
  if (C == nullptr && any) return -14;
  if (ldc < std::max(1, m)) return -15;
  if (too_long(m, n, q, groups)) return OZGEMM_RANGE;
  const size_t size = elem_bytes(type);
  const size_t cb = extent(m, n, ldc, 0, 1, elem_bytes(ctype));
  if (any && (overlap(C, cb, A, extent(ar, ac, lda, stridea, groups, size)) ||
              overlap(C, cb, B, extent(q, n, ldb, 0, 1, size)) ||
              overlap(C, cb, offsets, ((size_t)groups + 1) * 4)))
    return -14;
  const Rooms r = gemm_rooms(type, groups, m, n, q, transa, A, lda, stridea, B, ldb);
  if (r.total > 0 && (workspace == nullptr || ((uintptr_t)workspace & (WS_ALIGN - 1)))) return -16;
  if (workspace_bytes < r.total) return OZGEMM_WORKSPACE_TOO_SMALL;
  if (!any) return OZGEMM_OK;

  hipStream_t st = (hipStream_t)hip_stream;
  char* ws = (char*)workspace;
  Grouped16 g{};
  g.bf16 = type == OZGEMM_BF16;
  g.f32 = type == OZGEMM_F32;
  g.m = m;
  g.n = n;
  g.q = q;
  g.groups = groups;
  g.offsets = offsets;
  g.C = C;
  g.ctype = ctype;
  g.ldc = ldc;
  g.few = r.few > 0;
  g.edge = r.edge;
  g.parts = r.parts;
  g.partial = (float*)(ws + r.partial);
  // (F32 operands stay here for few columns, or where nothing is read)
  g.A = in_place(A, lda, (long)stridea, transa == 0 && (g.few || !g.f32), ar);
  g.B = in_place(B, ldb, 0, false, q);
  if (!grouped_n_fits(g)) return OZGEMM_RANGE;
  if (r.A.used) {
    g.A = sliced(type, r.A, ws, (long)m * r.A.ld, m);
    uint16_t* d = (uint16_t*)(ws + r.A.at);
    int32_t* ex = (int32_t*)(ws + r.A.ex);
    if (transa)
      OZ_TRY(launch_slice_rows(type, A, lda, (long)stridea, groups, m, q, d, r.A.ld, (long)r.A.plane, ex, st));
    else
      OZ_TRY(launch_slice_cols(type, A, lda, (long)stridea, groups, m, q, d, r.A.ld, (long)r.A.plane, ex,
                               (uint32_t*)(ws + r.A.part), st));
  }
  if (r.B.used) {
    g.B = sliced(type, r.B, ws, 0, 0);
    OZ_TRY(launch_slice_rows(type, B, ldb, 0, 1, n, q, (uint16_t*)(ws + r.B.at), r.B.ld, (long)r.B.plane,
                             (int32_t*)(ws + r.B.ex), st));
  }
  OZ_TRY(launch_grouped_n(g, st));
  return OZGEMM_OK;
}

size_t ozgemm_grouped_outer_workspace_bytes(int type, int groups, int m, int q, int n, const void* A, int lda,
                                            const void* B, int ldb) {
  if (!known_type(type) || groups < 0 || m < 0 || n < 0 || q < 0 || too_long(m, n, q, groups)) return 0;
  return outer_rooms(type, groups, m, q, n, A, lda, B, ldb).total;
}

int ozgemm_grouped_outer(int type, int ctype, int groups, int m, int q, int n, const void* A, int lda, const void* B,
                         int ldb, const int32_t* offsets, void* C, int ldc, long long stridec, void* workspace,
                         size_t workspace_bytes, void* hip_stream) {
  if (!known_type(type)) return -1;
  if (ctype != type && ctype != OZGEMM_F32) return -2;
  if (groups < 0) return -3;
  if (m < 0) return -4;
  if (q < 0) return -5;
  if (n < 0) return -6;
  const bool any = m > 0 && q > 0 && groups > 0;
  if (A == nullptr && any && n > 0) return -7;
  if (lda < std::max(1, m)) return -8;
  if (B == nullptr && any && n > 0) return -9;
  if (ldb < std::max(1, q)) return -10;
  if (offsets == nullptr && any) return -11;
  if (C == nullptr && any) return -12;
  if (ldc < std::max(1, m)) return -13;
  if (stridec < 0 || (any && groups > 1 && stridec < (long long)ldc * q)) return -14;
  if (too_long(m, n, q, groups)) return OZGEMM_RANGE;
  const size_t size = elem_bytes(type);
  const size_t cb = extent(m, q, ldc, stridec, groups, elem_bytes(ctype));
  if (any && (overlap(C, cb, A, extent(m, n, lda, 0, 1, size)) || overlap(C, cb, B, extent(q, n, ldb, 0, 1, size)) ||
              overlap(C, cb, offsets, ((size_t)groups + 1) * 4)))
    return -12;
  const Rooms r = outer_rooms(type, groups, m, q, n, A, lda, B, ldb);
  if (r.A.used && r.A.ld > LD16_MAX) return OZGEMM_RANGE;
  if (r.total > 0 && (workspace == nullptr || ((uintptr_t)workspace & (WS_ALIGN - 1)))) return -15;
  if (workspace_bytes < r.total) return OZGEMM_WORKSPACE_TOO_SMALL;
  if (!any) return OZGEMM_OK;

  hipStream_t st = (hipStream_t)hip_stream;
  char* ws = (char*)workspace;
  Grouped16 g{};
  g.bf16 = type == OZGEMM_BF16;
  g.f32 = type == OZGEMM_F32;
  g.m = m;
  g.n = n;
  g.q = q;
  g.groups = groups;
  g.offsets = offsets;
  g.C = C;
  g.ctype = ctype;
  g.ldc = ldc;
  g.cbatch = (long)stridec;
  g.parts = r.parts;
  g.partial = (float*)(ws + r.partial);
  g.few = r.few > 0;
  g.edge = r.edge;
  g.A = in_place(A, lda, 0, g.few || !g.f32, m);
  g.B = in_place(B, ldb, 0, g.few || !g.f32, q);
  if (!grouped_k_fits(g)) return OZGEMM_RANGE;
  if (r.A.used) {  // then B's too
    g.A = sliced(type, r.A, ws, 0, m);
    g.B = sliced(type, r.B, ws, 0, q);
    OZ_TRY(launch_slice_groups(type, A, lda, m, n, offsets, groups, (uint16_t*)(ws + r.A.at), r.A.ld,
                               (long)r.A.plane, (int32_t*)(ws + r.A.ex), (uint32_t*)(ws + r.A.part), st));
    OZ_TRY(launch_slice_groups(type, B, ldb, q, n, offsets, groups, (uint16_t*)(ws + r.B.at), r.B.ld,
                               (long)r.B.plane, (int32_t*)(ws + r.B.ex), (uint32_t*)(ws + r.B.part), st));
  }
  OZ_TRY(launch_grouped_k(g, st));
  return OZGEMM_OK;
}

}  // extern "C"
