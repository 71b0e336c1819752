// Blocks of 128 in 8 bits (block8.h), of a matrix, of its transpose, or of
// both from one reading.
//
//   rows = 1:    a scale for every row and 128 columns   (transpose: for every column and 128 rows)
//   rows = 128:  a scale for every 128 x 128 tile
//
// A block of threads takes one 128 x 128 tile into registers: thread (rg, cg)
// its rows 8 rg .. + 7 and columns 8 cg .. + 7, eight 16-byte loads (twice as
// many in F32), all in flight before the first is used.  Row maxima meet in 16
// neighbouring lanes, column maxima in LDS, where the transposed bytes are
// turned too, so that both results leave in whole lines.
//
// Bound by HBM: 16384 x 4096 of BF16, both results, 57 us or 4.7 TB/s, one result 38 us
// or 5.2 (a large copy: 4.9); 4096 x 8192 of F32, both, 34 us where the caches hold a part of it.
// With registers for four blocks a compute unit instead of three some of the tile went to scratch
// memory (38 us became 65).  Turning costs two thirds of LDS's cycles in bank conflicts, which the
// loads hide: pieces laid out without any took as long.
#include <algorithm>

#include "block8.h"
#include "oz_internal.h"
#include "products.h"

namespace oz {
namespace {

struct Result8 {
  uint8_t* v;  // nullptr: not asked for
  long ld;
  float* s;
  long srow, sblock;  // of scale (row, block)
};

struct Quantize {
  const void* x;
  long ld;
  int n, q, tiles_q;  // rows, entries of a row
  Result8 plain, turned;
};

template <int TYPE, int QTYPE, int ROWS>
__global__ __launch_bounds__(256) void quantize_kernel(Quantize g) {
  constexpr int PITCH = BLOCK8 + 8;  // bytes: 8 lanes' 8-byte pieces of one column group fall in different banks
  __shared__ __attribute__((aligned(16))) uint8_t turn[BLOCK8 * PITCH];
  __shared__ uint32_t colmax[BLOCK8], tilemax;
  const int t = threadIdx.x, rg = t >> 4, cg = t & 15;
  const int tr = blockIdx.x / g.tiles_q, tc = blockIdx.x % g.tiles_q;
  const int row0 = tr * BLOCK8 + rg * 8, col0 = tc * BLOCK8 + cg * 8;
  const int cols = g.q - col0;
  if (ROWS != 1 || g.turned.v != nullptr) {
    if (t < BLOCK8) colmax[t] = 0;
    if (t == 0) tilemax = 0;
    __syncthreads();
  }
  Raw8<TYPE> raw[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (row0 + r < g.n && cols > 0)
      raw[r].load(g.x, (long)(row0 + r) * g.ld + col0, cols);
    else
      raw[r].zero();
  }
  uint32_t rmax[8], cmax[8] = {};
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    rmax[r] = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t a = finite_abs(raw[r].get(c));
      rmax[r] = max(rmax[r], a);
      cmax[c] = max(cmax[c], a);
    }
  }
  int tile_e = 0;
  if (ROWS != 1) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) m = max(m, rmax[r]);
    m = max16(m);
    if (cg == 0) atomicMax(&tilemax, m);  // (integers: in any order the same)
    __syncthreads();
    tile_e = scale_exponent<QTYPE>(tilemax);
  }
  if (g.plain.v != nullptr) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int e = ROWS == 1 ? scale_exponent<QTYPE>(max16(rmax[r])) : tile_e;
      if (row0 + r < g.n && cols > 0) {
        const float f = power_of_two(-e);
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = no_inf(raw[r].get(c)) * f;
        const v2u b = {Eight<QTYPE>::pack4(v[0], v[1], v[2], v[3]), Eight<QTYPE>::pack4(v[4], v[5], v[6], v[7])};
        store_bytes(g.plain.v + (long)(row0 + r) * g.plain.ld + col0, b, cols);
        if (ROWS == 1 && cg == 0) g.plain.s[(row0 + r) * g.plain.srow + tc * g.plain.sblock] = power_of_two(e);
      }
    }
    if (ROWS != 1 && t == 0) g.plain.s[tr * g.plain.srow + tc * g.plain.sblock] = power_of_two(tile_e);
  }
  if (g.turned.v == nullptr) return;
  int ce[8];
  if (ROWS == 1) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t m = cmax[c];  // of the wavefront's four row groups, then of all
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if ((t & 48) == 0) atomicMax(&colmax[cg * 8 + c], m);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 8; ++c) ce[c] = scale_exponent<QTYPE>(colmax[cg * 8 + c]);
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) ce[c] = tile_e;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float f = power_of_two(-ce[c]);
    float v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = no_inf(raw[r].get(c)) * f;
    *reinterpret_cast<v2u*>(turn + (cg * 8 + c) * PITCH + rg * 8) =
        v2u{Eight<QTYPE>::pack4(v[0], v[1], v[2], v[3]), Eight<QTYPE>::pack4(v[4], v[5], v[6], v[7])};
  }
  __syncthreads();
  // column c of the tile is a row of the result: 16 lanes write its 128 bytes
  const int rows = g.n - tr * BLOCK8 - cg * 8;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int c = p * 16 + rg, col = tc * BLOCK8 + c;
    if (col >= g.q || rows <= 0) continue;
    store_bytes(g.turned.v + (long)col * g.turned.ld + tr * BLOCK8 + cg * 8,
                *reinterpret_cast<const v2u*>(turn + c * PITCH + cg * 8), rows);
  }
  if (ROWS == 1) {
    const int col = tc * BLOCK8 + t;
    if (t < BLOCK8 && col < g.q)
      g.turned.s[col * g.turned.srow + tr * g.turned.sblock] = power_of_two(scale_exponent<QTYPE>(colmax[t]));
  } else if (t == 0) {
    g.turned.s[tc * g.turned.srow + tr * g.turned.sblock] = power_of_two(tile_e);
  }
}

template <int TYPE, int QTYPE>
void launch_rows(int rows, const Quantize& g, unsigned blocks, hipStream_t st) {
  if (rows == 1)
    quantize_kernel<TYPE, QTYPE, 1><<<blocks, 256, 0, st>>>(g);
  else
    quantize_kernel<TYPE, QTYPE, BLOCK8><<<blocks, 256, 0, st>>>(g);
}

template <int TYPE>
void launch_type(int qtype, int rows, const Quantize& g, unsigned blocks, hipStream_t st) {
  if (qtype == OZGEMM_E4M3)
    launch_rows<TYPE, OZGEMM_E4M3>(rows, g, blocks, st);
  else
    launch_rows<TYPE, OZGEMM_E5M2>(rows, g, blocks, st);
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" int ozgemm_quantize_blocks(int type, int qtype, int rows, int n, int q, const void* X, int ldx, void* V,
                                      int ldv, float* S, long long srow, long long sblock, void* Vt, int ldvt,
                                      float* St, long long strow, long long stblock, void* hip_stream) {
  if (type != OZGEMM_F32 && type != OZGEMM_BF16 && type != OZGEMM_F16) return -1;
  if (qtype != OZGEMM_E4M3 && qtype != OZGEMM_E5M2) return -2;
  if (rows != 1 && rows != BLOCK8) return -3;
  if (n < 0) return -4;
  if (q < 0) return -5;
  const bool any = n > 0 && q > 0;
  if (X == nullptr && any) return -6;
  if (ldx < std::max(1, q)) return -7;
  if (V == nullptr && Vt == nullptr && any) return -8;
  if (V != nullptr) {
    if (ldv < std::max(1, q)) return -9;
    if (S == nullptr && any) return -10;
    if (srow < 0) return -11;
    if (sblock < 0) return -12;
  }
  if (Vt != nullptr) {
    if (ldvt < std::max(1, n)) return -14;
    if (St == nullptr && any) return -15;
    if (strow < 0) return -16;
    if (stblock < 0) return -17;
  }
  if (n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return OZGEMM_RANGE;
  if (!any) return OZGEMM_OK;
  const size_t xb = extent(q, n, ldx, 0, 1, elem_bytes(type));
  const size_t vb = V ? extent(q, n, ldv, 0, 1, 1) : 0, vtb = Vt ? extent(n, q, ldvt, 0, 1, 1) : 0;
  const size_t rb = (n - 1) / rows, qb = (q - 1) / BLOCK8;  // last row and block of the scales
  const size_t sb = V ? (rb * srow + qb * sblock + 1) * sizeof(float) : 0;
  const size_t stb = Vt ? ((q - 1) / rows * (size_t)strow + (n - 1) / BLOCK8 * (size_t)stblock + 1) * sizeof(float) : 0;
  if (V && !places_differ((n - 1) / rows + 1, (q - 1) / BLOCK8 + 1, srow, sblock)) return -11;
  if (Vt && !places_differ((q - 1) / rows + 1, (n - 1) / BLOCK8 + 1, strow, stblock)) return -16;
  if (overlap(V, vb, X, xb)) return -8;
  if (overlap(S, sb, X, xb) || overlap(S, sb, V, vb)) return -10;
  if (overlap(Vt, vtb, X, xb) || overlap(Vt, vtb, V, vb) || overlap(Vt, vtb, S, sb)) return -13;
  if (overlap(St, stb, X, xb) || overlap(St, stb, V, vb) || overlap(St, stb, S, sb) || overlap(St, stb, Vt, vtb))
    return -15;
  const long tiles_q = (q + BLOCK8 - 1) / BLOCK8, tiles = tiles_q * ((n + BLOCK8 - 1) / BLOCK8);
  if (tiles > (1L << 24) - 1) return OZGEMM_RANGE;  // 2^32 threads of a launch
  const Quantize g{X, ldx, n, q, (int)tiles_q, Result8{(uint8_t*)V, ldv, S, (long)srow, (long)sblock},
                   Result8{(uint8_t*)Vt, ldvt, St, (long)strow, (long)stblock}};
  hipStream_t st = (hipStream_t)hip_stream;
  if (type == OZGEMM_F32)
    launch_type<OZGEMM_F32>(qtype, rows, g, (unsigned)tiles, st);
  else if (type == OZGEMM_BF16)
    launch_type<OZGEMM_BF16>(qtype, rows, g, (unsigned)tiles, st);
  else
    launch_type<OZGEMM_F16>(qtype, rows, g, (unsigned)tiles, st);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}
