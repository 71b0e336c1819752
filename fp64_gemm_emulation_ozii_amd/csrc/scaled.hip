// Host side of the products in scaled blocks: argument checks, aligned copies
// of operands off the 16-byte grid, and the launch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block8.h"
#include "gemm8.h"
#include "products.h"

namespace oz {
namespace {

constexpr size_t WS_ALIGN = 256;

bool known8(int type) { return type == OZGEMM_E4M3 || type == OZGEMM_E5M2; }

// Read in place: whole 16-byte pieces of every row, the last of which may end
// behind the row, inside the same aligned 16 bytes.
bool aligned8(const void* p, long ld) { return ((uintptr_t)p & 15) == 0 && ld % 16 == 0 && ld <= LD8_MAX; }

// The leading dimension of rows of q entries; one row alone has none, and takes that of rows laid out here.
long ld8(int rows, long ld, int q) { return rows == 1 ? (long)up(q, 16) : ld; }

// How the scales of one operand lie.
struct Scales {
  int rows, per;
  long long srow, sblock;
};

struct Rooms {
  bool a, b;    // copied
  bool sa, sb;  // scales turned over
  size_t a_at, b_at, sa_at, sb_at, partial, total;
  long ld;
  int parts;
};

// A tile loads its rows' scales of one block at a time: a line for each where
// they lie block after block of a row.  Turning them over first costs a launch
// (3 us), which pays where many tiles read them (8192 x 8192 x 4096: 288 us as
// they lie, 250 so).
bool turns(const Scales& s, int m, int n, int q) {
  return s.per == 1 && s.srow != 1 && s.rows > 1 && q > BLOCK8 && scaled_big(m, n, q);
}

Rooms rooms(int m, int n, int q, const void* A, int lda, const Scales& sa, const void* B, int ldb,
            const Scales& sb) {
  Rooms r{};
  r.parts = 1;
  if (m < 1 || n < 1 || q < 1) return r;
  r.ld = (long)up(q, 16);
  r.a = !aligned8(A, ld8(m, lda, q));
  r.b = !aligned8(B, ld8(n, ldb, q));
  r.sa = turns(sa, m, n, q);
  r.sb = turns(sb, m, n, q);
  const size_t blocks = (size_t)(q + BLOCK8 - 1) / BLOCK8;
  auto take = [&](bool wanted, size_t bytes) {
    const size_t at = r.total;
    if (wanted) r.total += up(bytes, WS_ALIGN);
    return at;
  };
  r.a_at = take(r.a, (size_t)m * r.ld);
  r.b_at = take(r.b, (size_t)n * r.ld);
  r.sa_at = take(r.sa, blocks * m * sizeof(float));
  r.sb_at = take(r.sb, blocks * n * sizeof(float));
  r.parts = scaled_parts(m, n, q);
  r.partial = take(r.parts > 1, (size_t)r.parts * m * n * sizeof(float));
  return r;
}

// Bytes from the first scale to the end of the last.
size_t scale_extent(int rows, int per, int q, long long srow, long long sblock) {
  if (rows < 1 || q < 1) return 0;
  return ((size_t)((rows - 1) / per) * (size_t)srow + (size_t)((q - 1) / BLOCK8) * (size_t)sblock + 1) * sizeof(float);
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozgemm_scaled_gemm_workspace_bytes(int m, int n, int q, const void* A, int lda, int rows_a,
                                          long long sarow, long long sablock, const void* B, int ldb, long long sbrow,
                                          long long sbblock) {
  if (m < 0 || n < 0 || q < 0 || m > OZGEMM_MAX_ROWS || n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return 0;
  return rooms(m, n, q, A, lda, Scales{m, rows_a, sarow, sablock}, B, ldb, Scales{n, 1, sbrow, sbblock}).total;
}

int ozgemm_scaled_gemm(int atype, int btype, int ctype, int m, int n, int q, const void* A, int lda, const float* SA,
                       int rows_a, long long sarow, long long sablock, const void* B, int ldb, const float* SB,
                       long long sbrow, long long sbblock, void* C, int ldc, void* workspace, size_t workspace_bytes,
                       void* hip_stream) {
  if (!known8(atype)) return -1;
  if (!known8(btype)) return -2;
  if (ctype != OZGEMM_F32 && ctype != OZGEMM_BF16 && ctype != OZGEMM_F16) return -3;
  if (m < 0) return -4;
  if (n < 0) return -5;
  if (q < 0) return -6;
  const bool any = m > 0 && n > 0;
  if (A == nullptr && any && q > 0) return -7;
  if (lda < std::max(1, q)) return -8;
  if (SA == nullptr && any && q > 0) return -9;
  if (rows_a != 1 && rows_a != BLOCK8) return -10;
  if (sarow < 0) return -11;
  if (sablock < 0) return -12;
  if (B == nullptr && any && q > 0) return -13;
  if (ldb < std::max(1, q)) return -14;
  if (SB == nullptr && any && q > 0) return -15;
  if (sbrow < 0) return -16;
  if (sbblock < 0) return -17;
  if (C == nullptr && any) return -18;
  if (ldc < std::max(1, m)) return -19;
  if (m > OZGEMM_MAX_ROWS || n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return OZGEMM_RANGE;
  if (!any) return OZGEMM_OK;
  const size_t cb = extent(m, n, ldc, 0, 1, elem_bytes(ctype));
  if (overlap(C, cb, A, extent(q, m, lda, 0, 1, 1)) || overlap(C, cb, B, extent(q, n, ldb, 0, 1, 1)) ||
      overlap(C, cb, SA, scale_extent(m, rows_a, q, sarow, sablock)) ||
      overlap(C, cb, SB, scale_extent(n, 1, q, sbrow, sbblock)))
    return -18;
  const Rooms r =
      rooms(m, n, q, A, lda, Scales{m, rows_a, sarow, sablock}, B, ldb, Scales{n, 1, sbrow, sbblock});
  if (r.total > 0 && (workspace == nullptr || ((uintptr_t)workspace & (WS_ALIGN - 1)))) return -20;
  if (workspace_bytes < r.total) return OZGEMM_WORKSPACE_TOO_SMALL;
  if (!scaled_fits(m, n, r.parts)) return OZGEMM_RANGE;

  hipStream_t st = (hipStream_t)hip_stream;
  char* ws = (char*)workspace;
  Scaled8 g{};
  g.A = Operand8{(const uint8_t*)A, ld8(m, lda, q), SA, (long)sarow, (long)sablock, rows_a == 1 ? 0 : 7};
  g.B = Operand8{(const uint8_t*)B, ld8(n, ldb, q), SB, (long)sbrow, (long)sbblock, 0};
  g.atype = atype;
  g.btype = btype;
  g.m = m;
  g.n = n;
  g.q = q;
  g.C = C;
  g.ctype = ctype;
  g.ldc = ldc;
  g.parts = r.parts;
  g.partial = (float*)(ws + r.partial);
  hipError_t e = hipSuccess;
  if (r.a) {
    e = launch_align_rows(g.A.p, lda, m, q, (uint8_t*)ws + r.a_at, r.ld, st);
    g.A.p = (const uint8_t*)ws + r.a_at;
    g.A.ld = r.ld;
  }
  if (e == hipSuccess && r.b) {
    e = launch_align_rows(g.B.p, ldb, n, q, (uint8_t*)ws + r.b_at, r.ld, st);
    g.B.p = (const uint8_t*)ws + r.b_at;
    g.B.ld = r.ld;
  }
  if (e == hipSuccess && r.sa) {
    e = launch_turn_scales(SA, g.A.srow, g.A.sblock, m, q, (float*)(ws + r.sa_at), st);
    g.A.s = (const float*)(ws + r.sa_at);
    g.A.srow = 1;
    g.A.sblock = m;
  }
  if (e == hipSuccess && r.sb) {
    e = launch_turn_scales(SB, g.B.srow, g.B.sblock, n, q, (float*)(ws + r.sb_at), st);
    g.B.s = (const float*)(ws + r.sb_at);
    g.B.srow = 1;
    g.B.sblock = n;
  }
  if (e == hipSuccess) e = launch_scaled(g, st);
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}

}  // extern "C"
