// Orthogonalisation by Newton-Schulz products:
//   X_0 = G / (|G|_F + eps),  P = X X^T,  Q = b P + c P^2,  X <- a X + Q X,
// X with its r rows no more than its c columns (G or its transpose; the
// iteration commutes with the transpose).
//
// X stays in half-precision slices (slices.hip) between the products:
// x 2^E = hi + lo with E from a bound on the singular values of each matrix's
// own iterate (scales.h), to 2^-22 or better, or 2^-38 of that bound for entries
// far below it, whatever the type and however small |G| is beside eps; P and Q
// lie likewise.  BF16, F16 and F32 all take three slice products of every two
// states.  (One product of the high slices alone, with P and Q in one slice, took
// half the time for BF16, but its results were off by 1.25 times their rounding
// on four layers of 1024 x 4096, by 2 after eight steps, and by 9 with schedules
// whose terms cancel, on matrices of low rank: so nothing takes it.)  F64 runs
// the library's Scheme II products.
//
// X stays as G lies: wide (r rows of c entries next to each other) or tall (c
// rows of r).  P = X X^T runs along the c entries, Q X along the r rows; the
// product kernel reads an operand K-contiguous or K-strided (tile16.h), so no
// transposed copy is kept.  P and P^2 are symmetric: tiles on and below the
// diagonal are computed and written twice.
#include <hip/hip_runtime.h>

#include <cmath>

#include "pieces.h"
#include "products.h"
#include "scales.h"
#include "step64.h"
#include "tile16.h"

namespace oz {

namespace {

__device__ __forceinline__ double load_value(const void* p, int type, long at) {
  switch (type) {
    case OZGEMM_F64: return ((const double*)p)[at];
    case OZGEMM_F32: return ((const float*)p)[at];
    case OZGEMM_BF16: return (float)((const __bf16*)p)[at];
    default: return (float)((const _Float16*)p)[at];
  }
}

__device__ __forceinline__ void store_value(void* p, int type, long at, double v) {
  switch (type) {
    case OZGEMM_F64: ((double*)p)[at] = v; break;
    case OZGEMM_F32: ((float*)p)[at] = (float)v; break;
    case OZGEMM_BF16: ((__bf16*)p)[at] = (__bf16)(float)v; break;
    default: ((_Float16*)p)[at] = (_Float16)(float)v; break;
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum of the block's values in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v, double* part) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((part[0] + part[1]) + (part[2] + part[3]));
}

// Eight entries next to each other.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, long at, int left, float (&v)[8]) {
  if (TYPE == OZGEMM_F32) {
    const float* q = (const float*)p + at;
    if (left >= 8) {
      *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f_any*>(q);
      *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f_any*>(q + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < left ? q[e] : 0.f;
    }
  } else {
    const short* q = (const short*)p + at;
    v8s h = {0, 0, 0, 0, 0, 0, 0, 0};
    if (left >= 8) {
      h = *reinterpret_cast<const v8s_any*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) h[e] = q[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = TYPE == OZGEMM_BF16 ? (float)__builtin_bit_cast(__bf16, (short)h[e])
                                 : (float)__builtin_bit_cast(_Float16, (short)h[e]);
  }
}

template <class V>
__device__ __forceinline__ void store8(void* p, int type, long at, int left, const V (&v)[8]) {
  if (type == OZGEMM_F32) {
    float* q = (float*)p + at;
    if (left >= 8) {
      *reinterpret_cast<v4f_any*>(q) = v4f{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<v4f_any*>(q + 4) = v4f{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) q[e] = v[e];
    }
    return;
  }
  v8s h;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    h[e] = type == OZGEMM_BF16 ? __builtin_bit_cast(short, (__bf16)v[e]) : __builtin_bit_cast(short, (_Float16)v[e]);
  short* q = (short*)p + at;
  if (left >= 8) {
    *reinterpret_cast<v8s_any*>(q) = h;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) q[e] = h[e];
  }
}

// Sums of squares in FP64 (no square of an FP32 value leaves its range):
// block (p, b) adds the pieces of 2048 entries p, p + parts, ... of matrix b's rows.
// Bound by reading G: 4096 x 8192 in bf16 takes 21.8 us, 3.1 TB/s.
template <int TYPE>
__global__ __launch_bounds__(256) void square_sum_kernel(const void* __restrict__ G, int rows, int cols, long ld,
                                                         long batch, double* __restrict__ part) {
  __shared__ double s[4];
  const long base = blockIdx.y * batch;
  const int per = (cols + 2047) / 2048, pieces = rows * per;
  // narrow rows: each wavefront takes a row of its own
  const bool narrow = cols <= 512;
  double sum = 0;
  const int first = narrow ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int step = narrow ? gridDim.x * 4 : gridDim.x;
  const int lane8 = (narrow ? (threadIdx.x & 63) : threadIdx.x) * 8;
  constexpr int AHEAD = TYPE == OZGEMM_F64 ? 1 : 4;  // pieces in flight
  for (int i0 = first; i0 < pieces; i0 += step * AHEAD) {
    float v[AHEAD][8];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u * step, r = i / per, c = (i - r * per) * 2048 + lane8;
      const int left = i < pieces ? cols - c : 0;
      if (TYPE == OZGEMM_F64) {
        const double* q = (const double*)G + base + r * ld + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) sum = __builtin_fma(q[e], q[e], sum);
      } else {
        load8<TYPE>(G, base + r * ld + c, left, v[u]);
      }
    }
    if (TYPE != OZGEMM_F64) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)v[u][e], (double)v[u][e], sum);
    }
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

hipError_t launch_square_sum(int type, const void* G, int rows, int cols, long ld, long batch, int batches, int parts,
                             double* part, hipStream_t st) {
  const dim3 g(parts, batches), t(256);
  switch (type) {
    case OZGEMM_F64: hipLaunchKernelGGL(square_sum_kernel<OZGEMM_F64>, g, t, 0, st, G, rows, cols, ld, batch, part); break;
    case OZGEMM_F32: hipLaunchKernelGGL(square_sum_kernel<OZGEMM_F32>, g, t, 0, st, G, rows, cols, ld, batch, part); break;
    case OZGEMM_BF16: hipLaunchKernelGGL(square_sum_kernel<OZGEMM_BF16>, g, t, 0, st, G, rows, cols, ld, batch, part); break;
    default: hipLaunchKernelGGL(square_sum_kernel<OZGEMM_F16>, g, t, 0, st, G, rows, cols, ld, batch, part);
  }
  return hipGetLastError();
}

// |G_b|_F from the partial sums of matrix b, in every thread of the block.
__device__ __forceinline__ double frobenius(const double* part, int parts, long b, double* s) {
  double v = 0;
  for (int i = threadIdx.x; i < parts; i += 256) v += part[b * parts + i];
  return sqrt(block_sum(v, s));
}

__device__ __forceinline__ double inverse_norm(const double* part, int parts, long b, double eps, double* s) {
  return 1.0 / (frobenius(part, parts, b, s) + eps);
}

__device__ __forceinline__ void split(float y, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)y;
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, (_Float16)(y - (float)h));
}

__device__ __forceinline__ float joined(uint16_t hi, uint16_t lo) {
  return (float)__builtin_bit_cast(_Float16, hi) + (float)__builtin_bit_cast(_Float16, lo);
}

// The factors of a matrix's products, which the kernels of every step read
// from the workspace: [step][matrix].
struct StepFactors {
  Factors of;
  int pad;
};
static_assert(sizeof(StepFactors) == 32, "two 16-byte words");

// G (rows x cols) scaled and cut into slices, zeros in the padding; one more
// block for each matrix works out the factors of its steps meanwhile.  Bound by
// HBM: 4096 x 8192 in bf16 reads 67 MB and writes 134 in 52.8 us, 3.8 TB/s.
constexpr int PREPARE_RUNS = 4;  // runs of 8 entries per thread, at most

struct Prepare {
  const void* G;
  int rows, cols;
  long ld, batch;
  const double* part;
  int parts;
  double eps;
  uint16_t* X;   // [batch][2][rows_pad][cols_pad]
  int rows_pad, cols_pad;
  int each;      // runs per thread: fewer where the blocks would not fill the card
  StepFactors* factors;
  int steps, batches;
  double co[3 * OZGEMM_ORTHO_STEPS_MAX];
};

template <int TYPE>
__global__ __launch_bounds__(256) void prepare_kernel(Prepare p) {
  __shared__ double s[4];
  const long b = blockIdx.y;
  const double norm = frobenius(p.part, p.parts, b, s), t0 = first_bound(norm, p.eps);
  if (blockIdx.x == gridDim.x - 1) {
    __shared__ Bends bends[OZGEMM_ORTHO_STEPS_MAX];
    if ((int)threadIdx.x < p.steps) {
      const double* co = p.co + 3 * threadIdx.x;
      bends[threadIdx.x] = bends_of(co[0], co[1], co[2]);
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    double t = t0;
    for (int k = 0; k < p.steps; ++k) {
      const Bounds r = advance(bends[k], t);
      p.factors[(long)k * p.batches + b].of = factors_of(bends[k], r);
      t = r.next;
    }
    return;
  }
  const double f = 1.0 / (norm + p.eps) * ldexp(1.0, grid_exponent(t0));
  const long plane = (long)p.rows_pad * p.cols_pad, base = b * p.batch;
  const int per = p.cols_pad / 8, runs = (int)(plane / 8);
#pragma unroll
  for (int i = 0; i < PREPARE_RUNS; ++i) {
    const int at = (blockIdx.x * p.each + i) * 256 + threadIdx.x;
    if (i >= p.each || at >= runs) return;
    const int r = at / per, c = (at - r * per) * 8;
    float v[8];
    load8<TYPE>(p.G, base + r * p.ld + c, r < p.rows ? p.cols - c : 0, v);
    v8s h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint16_t hi, lo;
      split((float)(v[e] * f), hi, lo);
      if (r >= p.rows || c + e >= p.cols) hi = lo = 0;  // (0 f is NaN where the norm is)
      h[e] = (short)hi;
      l[e] = (short)lo;
    }
    uint16_t* out = p.X + b * 2 * plane + (long)at * 8;
    *reinterpret_cast<v8s*>(out) = h;
    *reinterpret_cast<v8s*>(out + plane) = l;
  }
}

__global__ __launch_bounds__(256) void normalise_kernel(const void* G, int type, int rows, int cols, long ld,
                                                        long batch, const double* __restrict__ part, int parts,
                                                        double eps, void* O, long ldo, long batcho, long first) {
  __shared__ double s[4];
  const long b = blockIdx.y;
  const double f = inverse_norm(part, parts, b, eps, s);
  const long at = (first + blockIdx.x) * 256 + threadIdx.x;
  if (at >= (long)rows * cols) return;
  const long r = at / cols, c = at - r * cols;
  store_value(O, type, b * batcho + r * ldo + c, load_value(G, type, b * batch + r * ld + c) * f);
}

// One product of a step: D = A B^T on padded planes, then
// v = alpha D + beta S, rounded to slices of N ([j][i]; a symmetric result is
// computed on and below the diagonal and written on both sides of it) or, in
// the last step, to the result.
struct Step {
  const uint16_t* A;  // [batch] a_batch apart, two slices a_plane apart
  const uint16_t* B;
  long a_batch, a_plane, b_batch, b_plane;
  int a_ld, b_ld;
  int m, n, k;        // padded
  int batch;
  const StepFactors* factors;  // of this step; v = f[which] D + g[which] S
  int which;
  const uint16_t* S;  // like N; nullptr: none
  uint16_t* N;
  long s_batch, s_plane;  // of S and N alike
  void* O;
  int otype;
  long ldo, batcho;
  int om, on;         // the result's own size
};

// The tile with corner (m0, n0) of matrix b; sizes are multiples of 64, and
// what lies past them arrives as zero and is not written.
template <class Tile, bool AKS, bool BKS, bool SYM>
__device__ __forceinline__ void step_tile(const Step& p, char* smem, long b, int m0, int n0) {
  const Source16 A{p.A + b * p.a_batch + (AKS ? (long)m0 : (long)m0 * p.a_ld), p.a_plane, p.a_ld, p.m - m0,
                   AKS ? p.m - m0 : p.k};
  const Source16 B{p.B + b * p.b_batch + (BKS ? (long)n0 : (long)n0 * p.b_ld), p.b_plane, p.b_ld, p.n - n0,
                   BKS ? p.n - n0 : p.k};
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, A, B, p.k);

  // Each wavefront passes its accumulators 16 columns at a time through a
  // piece of LDS of its own; a lane then holds runs of 8 rows.  S's runs for
  // the next 16 columns are on their way meanwhile.
  constexpr int WTM = Tile::FM * 16, PITCH = WTM + 4, RUNS = WTM / 8, CH = (16 * RUNS + 63) / 64;
  static_assert(16 * RUNS % 64 == 0, "whole wavefronts of runs");
  static_assert(Tile::NW * 16 * PITCH * 4 <= Tile::SMEM, "staging fits the operand buffers");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* stage = reinterpret_cast<float*>(smem) + wave * 16 * PITCH;
  const int mw = m0 + Tile::wave_m(wave) * WTM, nw = n0 + Tile::wave_n(wave) * (Tile::FN * 16);
  const uint16_t* S = p.S ? p.S + b * p.s_batch : nullptr;
  uint16_t* N = p.N + b * p.s_batch;
  const bool mirror = SYM && m0 != n0;  // a diagonal tile holds both halves itself
  auto offset = [&](int j, int ch) {
    const int at = ch * 64 + lane;
    return (long)(nw + j * 16 + at / RUNS) * p.m + mw + at % RUNS * 8;
  };
  // (a run of 8 rows and 16 columns lie inside or outside as a whole)
  auto inside = [&](int j, int ch) { return nw + j * 16 < p.n && mw + (ch * 64 + lane) % RUNS * 8 < p.m; };
  const Factors& by = p.factors[b].of;
  const float alpha = by.f[p.which], beta = by.g[p.which];
  const int down = by.next;  // the result itself is on no grid
  v8s sh[2][CH] = {}, sl[2][CH] = {};
  auto fetch = [&](int j) {
    if (S == nullptr) return;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      if (!inside(j, ch)) continue;
      const long off = offset(j, ch);
      sh[j & 1][ch] = *reinterpret_cast<const v8s*>(S + off);
      sl[j & 1][ch] = *reinterpret_cast<const v8s*>(S + p.s_plane + off);
    }
  };
  fetch(0);
  slice_barrier<0>();  // every wave has read its last operands, and no load into LDS is in flight
#pragma unroll
  for (int j = 0; j < Tile::FN; ++j) {
    if (j + 1 < Tile::FN) fetch(j + 1);
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
      *reinterpret_cast<v4f*>(stage + (lane & 15) * PITCH + i * 16 + 4 * (lane >> 4)) = acc[i][j];
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      const int at = ch * 64 + lane, c = at / RUNS, r = at % RUNS * 8;
      if (!inside(j, ch)) continue;
      float v[8];
      *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r);
      *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = __builtin_fmaf(beta, joined((uint16_t)sh[j & 1][ch][e], (uint16_t)sl[j & 1][ch][e]), v[e] * alpha);
      if (!SYM && p.O != nullptr) {
        const int col = nw + j * 16 + c, row = mw + r;
        if (col < p.on) {
          const long to = b * p.batcho + (long)col * p.ldo + row;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], -down);
          store8(p.O, p.otype, to, p.om - row, v);
        }
        continue;
      }
      v8s h, l;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint16_t hi, lo;
        split(v[e], hi, lo);
        h[e] = (short)hi;
        l[e] = (short)lo;
      }
      const long off = offset(j, ch);
      *reinterpret_cast<v8s*>(N + off) = h;
      *reinterpret_cast<v8s*>(N + p.s_plane + off) = l;
      // the rounded slices go back to the staging piece for the other side
      if (mirror) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint32_t*>(stage)[c * PITCH + r + e] = (uint16_t)h[e] | ((uint32_t)(uint16_t)l[e] << 16);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
    if (mirror) {  // 16 columns of one row: 32 bytes
#pragma unroll
      for (int ch = 0; ch < (WTM * 2 + 63) / 64; ++ch) {
        const int at = ch * 64 + lane, r = at >> 1, c = (at & 1) * 8;
        if (r >= WTM || mw + r >= p.m || nw + j * 16 >= p.n) continue;
        v8s h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = reinterpret_cast<const uint32_t*>(stage)[(c + e) * PITCH + r];
          h[e] = (short)x;
          l[e] = (short)(x >> 16);
        }
        const long off = (long)(mw + r) * p.n + nw + j * 16 + c;
        *reinterpret_cast<v8s*>(N + off) = h;
        *reinterpret_cast<v8s*>(N + p.s_plane + off) = l;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
      asm volatile("" ::: "memory");
    }
  }
}

// One block per tile; the tiles past `whole` (a last round of them that would
// leave most compute units idle) are cut into quarters.  (Blocks that walk
// tiles, as the grouped products', gained nothing here: a matrix has few
// rounds, and a step's epilogue reads and writes as much as its operands.)
// Bound by the matrix cores where the tiles fill the card (4096 x 8192: Q X 706 us,
// 389 TFLOPS or 1170 of its slices, 63% of the MFMA cycles at the 1.74 GHz that
// the power leaves; X X^T about 400 us, 1030 of its slices).  Q X of four 1024 x
// 4096 takes 107 us (960 of its slices): four rounds of tiles whose loads and
// stores (200 MB) do not overlap their products.
template <int BT, int WM, int WN, int NB, bool QUARTERS, bool AKS, bool BKS, bool SYM>
__global__ __launch_bounds__(WM* WN * 64, 2) void step_kernel(Step p, int whole) {
  using Tile = Tile16<Half, BT, BT, WM, WN, AKS, BKS, NB, true>;
  using Small = Tile16<Half, QUARTERS ? BT / 2 : BT, QUARTERS ? BT / 2 : BT, WM, WN, AKS, BKS, 4, true>;
  constexpr int SMEM = QUARTERS && Small::SMEM > Tile::SMEM ? Small::SMEM : Tile::SMEM;
  __shared__ __attribute__((aligned(1024))) char smem[SMEM];
  const int tm = (p.m + BT - 1) / BT, tn = (p.n + BT - 1) / BT;
  const int per = SYM ? tm * (tm + 1) / 2 : tm * tn, total = per * p.batch;
  int L = blockIdx.x, quarter = -1;
  if (QUARTERS && L >= whole) {
    quarter = (L - whole) % 4;
    L = whole + (L - whole) / 4;
  }
  const int w = xcd_order(L, total);
  const long b = w / per;
  const int t = w % per;
  int mi, nj;
  if (SYM) {
    triangle_order<4>(t, tm, mi, nj);
  } else {
    panel_order<4>(t, tm, tn, mi, nj);
  }
  int m0 = mi * BT, n0 = nj * BT;
  if (QUARTERS && quarter >= 0) {
    m0 += (quarter & 1) * (BT / 2);
    n0 += (quarter >> 1) * (BT / 2);
    if (m0 >= p.m || n0 >= p.n || (SYM && m0 < n0)) return;
    step_tile<Small, AKS, BKS, SYM>(p, smem, b, m0, n0);
  } else {
    step_tile<Tile, AKS, BKS, SYM>(p, smem, b, m0, n0);
  }
}

template <int BT, int WM, int WN, int NB, bool QUARTERS>
hipError_t launch_step_t(const Step& p, bool aks, bool sym, int units, hipStream_t st) {
  const long tm = (p.m + BT - 1) / BT, tn = (p.n + BT - 1) / BT;
  const long tiles = (sym ? tm * (tm + 1) / 2 : tm * tn) * p.batch, rest = tiles % units;
  const int whole = (int)(QUARTERS && rest * 2 <= units ? tiles - rest : tiles);
  const dim3 grid((unsigned)(whole + 4 * (tiles - whole))), block(WM * WN * 64);
  if (sym && aks)
    hipLaunchKernelGGL((step_kernel<BT, WM, WN, NB, QUARTERS, true, true, true>), grid, block, 0, st, p, whole);
  else if (sym)
    hipLaunchKernelGGL((step_kernel<BT, WM, WN, NB, QUARTERS, false, false, true>), grid, block, 0, st, p, whole);
  else if (aks)
    hipLaunchKernelGGL((step_kernel<BT, WM, WN, NB, QUARTERS, true, false, false>), grid, block, 0, st, p, whole);
  else
    hipLaunchKernelGGL((step_kernel<BT, WM, WN, NB, QUARTERS, false, false, false>), grid, block, 0, st, p, whole);
  return hipGetLastError();
}

// The tile size of a product of S K slices: the modelled time, in us, of its
// rounds of one tile per compute unit (a quartered last round counts 0.4 per
// `units` quarters).  A round takes S slices and a start and an end; measured
// with every unit busy: 128 x 128  1.2 S + 8   64 x 64  0.43 S + 3
// (64 x 64: two blocks of four wavefronts on a unit; where there is only one for
// each, eight wavefronts and four buffers, 0.53 S against 0.74 S.)
hipError_t launch_step(const Step& p, bool aks, bool sym, hipStream_t st) {
  int units = 0;
  const hipError_t err = device_units(&units);
  if (err != hipSuccess) return err;
  const double S = p.k / BK16;
  auto rounds = [&](int bt, bool quarters) {
    const long tm = (p.m + bt - 1) / bt, tn = (p.n + bt - 1) / bt;
    const long tiles = (sym ? tm * (tm + 1) / 2 : tm * tn) * p.batch, rest = tiles % units;
    const double last = rest == 0 ? 0 : quarters && rest * 2 <= units ? 0.4 * ((4 * rest + units - 1) / units) : 1;
    return (double)(tiles / units) + last;
  };
  if (rounds(128, true) * (1.2 * S + 8) <= rounds(64, false) * (0.43 * S + 3))
    return launch_step_t<128, 2, 4, 2, true>(p, aks, sym, units, st);
  if (rounds(64, false) <= 1) return launch_step_t<64, 2, 4, 4, false>(p, aks, sym, units, st);
  return launch_step_t<64, 2, 2, 2, false>(p, aks, sym, units, st);
}

// P = X X^T for few rows and long ones, along the c entries in `parts` parts
// (five steps on one f32 matrix of 64 x 4096: 172 us in one part, 93 so):
// every block sums 64 x 64 entries over its part of the slices, and the
// parts' sums meet in FP32.  (All of P: at these sizes the time is a block's
// slices, not the operations.)
struct Parts {
  const uint16_t* X;
  long x_batch, x_plane;
  int x_ld, r, c, batch, parts;
  const StepFactors* factors;
  float* partial;  // [parts][batch][r][r]
  uint16_t* P;     // [batch][2][r][r]
};

template <bool KS>
__global__ __launch_bounds__(256, 2) void gram_parts_kernel(Parts p) {
  using Tile = Tile16<Half, 64, 64, 2, 2, KS, KS, 2, true>;
  __shared__ __attribute__((aligned(1024))) char smem[Tile::SMEM];
  const int t = p.r / 64;
  int w = blockIdx.x;
  const int part = w % p.parts;
  w /= p.parts;
  const int nj = w % t, mi = w / t % t;
  const long b = w / (t * t);
  const int slices = p.c / BK16, each = (slices + p.parts - 1) / p.parts;
  const int from = min(part * each, slices) * BK16, len = min(p.c - from, each * BK16);
  const uint16_t* X = p.X + b * p.x_batch;
  auto source = [&](int r0) {
    return Source16{X + (KS ? (long)from * p.x_ld + r0 : (long)r0 * p.x_ld + from), p.x_plane, p.x_ld, p.r - r0,
                    KS ? p.r - r0 : p.c - from};
  };
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, source(mi * 64), source(nj * 64), max(len, 0));
  slice_barrier<0>();  // no load into LDS outlives the block
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* out = p.partial + ((long)part * p.batch + b) * p.r * p.r;
#pragma unroll
  for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
      *reinterpret_cast<v4f*>(out + (long)(nj * 64 + Tile::wave_n(wave) * 32 + j * 16 + (lane & 15)) * p.r + mi * 64 +
                              Tile::wave_m(wave) * 32 + i * 16 + 4 * (lane >> 4)) = acc[i][j];
}

__global__ __launch_bounds__(256) void gram_join_kernel(Parts p) {
  const long plane = (long)p.r * p.r, at = ((long)blockIdx.x * 256 + threadIdx.x) * 8;
  const long b = blockIdx.y;
  if (at >= plane) return;
  const float alpha = p.factors[b].of.f[0];
  v4f v[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) v[e] = sum_parts(p.partial + b * plane + at + 4 * e, p.batch * plane, p.parts, 4);
  v8s h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint16_t hi, lo;
    split(v[e / 4][e % 4] * alpha, hi, lo);
    h[e] = (short)hi;
    l[e] = (short)lo;
  }
  uint16_t* out = p.P + b * 2 * plane + at;
  *reinterpret_cast<v8s*>(out) = h;
  *reinterpret_cast<v8s*>(out + plane) = l;
}

hipError_t launch_gram_parts(const Parts& p, bool ks, hipStream_t st) {
  const dim3 grid((unsigned)((long)(p.r / 64) * (p.r / 64) * p.batch * p.parts));
  if (ks)
    hipLaunchKernelGGL((gram_parts_kernel<true>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((gram_parts_kernel<false>), grid, dim3(256), 0, st, p);
  const long runs = ((long)p.r * p.r / 8 + 255) / 256;
  hipLaunchKernelGGL(gram_join_kernel, dim3((unsigned)runs, p.batch), dim3(256), 0, st, p);
  return hipGetLastError();
}

// Parts of the c entries for a batch of r x c (padded): where the tiles leave
// most of the card's 256 units idle and each walks many slices.
int gram_parts(int batch, int r, int c) {
  const long tiles = (long)(r / 64) * (r / 64) * batch, slices = c / BK16;
  const long parts = tiles > 128 ? 1 : slices / 4 < 512 / tiles ? slices / 4 : 512 / tiles;
  return slices < 12 || parts < 2 ? 1 : (int)(parts < 32 ? parts : 32);
}

// FP64: X and its transpose, Q = b P + c P2, X <- a X + Y both ways round
__global__ __launch_bounds__(256) void prepare64_kernel(const double* __restrict__ G, int rows, int cols, long ld,
                                                        const double* __restrict__ part, int parts, double eps,
                                                        double* __restrict__ X, double* __restrict__ XT) {
  __shared__ double s[4];
  __shared__ double tile[64][65];
  const double f = inverse_norm(part, parts, 0, eps, s);
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = r0 + (i >> 6), c = c0 + (i & 63);
    if (r < rows && c < cols) X[(long)r * cols + c] = tile[i >> 6][i & 63] = G[r * ld + c] * f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = c0 + (i >> 6), r = r0 + (i & 63);
    if (r < rows && c < cols) XT[(long)c * rows + r] = tile[i & 63][i >> 6];
  }
}

// X_0 of a batch, as G lies, on the way through the FP64 matrix cores
__global__ __launch_bounds__(256) void scale64_kernel(const double* __restrict__ G, int rows, int cols, long ld,
                                                      long batch, const double* __restrict__ part, int parts,
                                                      double eps, double* __restrict__ X) {
  __shared__ double s[4];
  const long b = blockIdx.y;
  const double f = inverse_norm(part, parts, b, eps, s);
  const long at = (long)blockIdx.x * 256 + threadIdx.x;
  if (at >= (long)rows * cols) return;
  const long r = at / cols, c = at - r * cols;
  X[b * rows * cols + at] = G[b * batch + r * ld + c] * f;
}

__global__ __launch_bounds__(256) void combine64_kernel(double* __restrict__ Q, const double* __restrict__ P, double b,
                                                        double c, long n) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) Q[i] = __builtin_fma(c, Q[i], b * P[i]);
}

// X (rows x cols, as it lies) <- a X + Y, with its transpose; the last step writes the result instead
__global__ __launch_bounds__(256) void update64_kernel(double* __restrict__ X, double* __restrict__ XT,
                                                       const double* __restrict__ Y, double a, int rows, int cols,
                                                       double* __restrict__ O, long ldo, int transpose) {
  __shared__ double tile[64][65];
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = r0 + (i >> 6), c = c0 + (i & 63);
    if (r >= rows || c >= cols) continue;
    const long at = (long)r * cols + c;
    const double v = __builtin_fma(a, X[at], Y[at]);
    if (O == nullptr)
      X[at] = v;
    else if (!transpose)
      O[r * ldo + c] = v;
    tile[i >> 6][i & 63] = v;
  }
  __syncthreads();
  if (O != nullptr && !transpose) return;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = c0 + (i >> 6), r = r0 + (i & 63);
    if (r >= rows || c >= cols) continue;
    if (O != nullptr)
      O[c * ldo + r] = tile[i & 63][i >> 6];
    else
      XT[(long)c * rows + r] = tile[i & 63][i >> 6];
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int SQUARE_PARTS = 256;

// Blocks that sum one matrix's squares: up to two pieces of a row per
// wavefront (narrow rows) or block, SQUARE_PARTS at most.
int square_parts(int m, int n) {  // n rows of m entries
  const long pieces = m <= 512 ? (n + 7) / 8 : ((long)n * ((m + 2047) / 2048) + 1) / 2;
  return (int)(pieces < 1 ? 1 : pieces > SQUARE_PARTS ? SQUARE_PARTS : pieces);
}

struct OrthoLayout {
  int rp, cp;  // sizes padded to 64
  int parts;   // of P = X X^T
  size_t partial;
  size_t part, factors, X1, X2, P, Q, total;  // 16-bit slices
  bool direct;                             // FP64: by the FP64 matrix cores
  size_t X, XT, Y, dgemm;                  // FP64
};

// Whether an FP64 batch goes by the FP64 matrix cores (step64.h) or by Scheme
// II products, from modelled times of a step in us.  A product of the former
// takes 1.2 us for every 64 of its inner dimension and 6 besides, or its
// operations (half of them for the symmetric results) at 30 TFLOPS.  Scheme II
// takes the matrices one after the other, 38 us per product for its passes'
// launches, s int8 products at 2.2 POP/s, and residues and results at 6 TB/s.
// Measured, five steps, s = 14, matrix cores against Scheme II, in ms:
//   512^2 0.29 / 0.64   520 x 3688 0.95 / 1.15   1024^2 0.91 / 0.90
//   1024 x 4096 2.3 / 1.6   2048^2 4.5 / 2.9   15 of 40 x 315 0.15 / 7.4
bool by_matrix_cores(int batch, int r, int c, int s) {
  const double R = r, C = c, B = batch;
  auto product = [&](double ops, double k) { return fmax(B * ops / 30e6, ceil(k / 64) * 1.2 + 6); };
  const double direct = product(R * R * C, C) + product(R * R * R, R) + product(2 * R * R * C, R);
  const double bytes = (16 + s) * (2 * R * C + 2 * R * R) + (8 + s) * (2 * R * R + R * C) + 32 * R * R + 32 * R * C;
  return direct <= B * (3 * 38 + s * 2 * (2 * R * R * C + R * R * R) / 2.2e9 + bytes / 6e6);
}

OrthoLayout ortho_layout(int type, int batch, int m, int n, int s) {
  OrthoLayout L{};
  const int r = m < n ? m : n, c = m < n ? n : m;
  auto take = [&](size_t bytes) {
    const size_t at = L.total;
    L.total += up(bytes, 256);
    return at;
  };
  L.part = take((size_t)batch * SQUARE_PARTS * 8);
  if (type == OZGEMM_F64) {
    const size_t rc = (size_t)r * c * 8, rr = (size_t)r * r * 8;
    L.direct = by_matrix_cores(batch, r, c, s);
    if (L.direct) {
      L.X = take(batch * rc);
      L.Y = take(batch * rc);
      L.P = take(batch * rr);
      L.Q = take(batch * rr);
      return L;
    }
    L.X = take(rc);
    L.XT = take(rc);
    L.Y = take(rc);
    L.P = take(rr);
    L.Q = take(rr);
    L.dgemm = take(dgemm_region_bytes(r, c, s));
    return L;
  }
  L.rp = (int)up(r, 64);
  L.cp = (int)up(c, 64);
  const size_t rc = (size_t)batch * 2 * L.rp * L.cp * 2, rr = (size_t)batch * 2 * L.rp * L.rp * 2;
  L.factors = take((size_t)batch * OZGEMM_ORTHO_STEPS_MAX * sizeof(StepFactors));
  L.X1 = take(rc);
  L.X2 = take(rc);
  L.P = take(rr);
  L.Q = take(rr);
  L.parts = gram_parts(batch, L.rp, L.cp);
  if (L.parts > 1) L.partial = take((size_t)L.parts * batch * L.rp * L.rp * 4);
  return L;
}

#define OZ_TRY(expr)                                                   \
  do {                                                                 \
    const hipError_t oz_err_ = (expr);                                 \
    if (oz_err_ != hipSuccess) return record_hip_error(oz_err_);       \
  } while (0)

// Whether no bound of a schedule's states leaves a double's sensible range, from t_0 = 1 on.
bool schedule_fits(const double* co, int steps) {
  double t = 1;
  for (int k = 0; k < steps; ++k) {
    const Bounds r = advance(bends_of(co[3 * k], co[3 * k + 1], co[3 * k + 2]), t);
    if (!in_range(r)) return false;
    t = r.next;
  }
  return true;
}

int ortho64(const OrthoLayout& L, int batch, int m, int n, const double* G, long ldg, long strideg, int steps,
            const double* co, double eps, int s, double* O, long ldo, long strideo, char* ws, hipStream_t st) {
  // G as it lies: n rows of m entries.  X: r x c column-major, i.e. c rows of r entries.
  const int r = m < n ? m : n, c = m < n ? n : m;
  const bool as_it_lies = r == m;  // c rows of r entries
  double* X = (double*)(ws + L.X);
  double* XT = (double*)(ws + L.XT);
  double* Y = (double*)(ws + L.Y);
  double* P = (double*)(ws + L.P);
  double* Q = (double*)(ws + L.Q);
  double* part = (double*)(ws + L.part);
  char* region = ws + L.dgemm;
  const dim3 tiles((m + 63) / 64, (n + 63) / 64), xt((r + 63) / 64, (c + 63) / 64);
  OZ_TRY(dgemm_region_table(region, s, st));
  for (int i = 0; i < batch; ++i) {
    const double* Gi = G + i * strideg;
    double* Oi = O + i * strideo;
    const int parts = square_parts(m, n);
    OZ_TRY(launch_square_sum(OZGEMM_F64, Gi, n, m, ldg, 0, 1, parts, part, st));
    hipLaunchKernelGGL(prepare64_kernel, tiles, dim3(256), 0, st, Gi, n, m, ldg, part, parts, eps,
                       as_it_lies ? X : XT, as_it_lies ? XT : X);
    OZ_TRY(hipGetLastError());
    for (int k = 0; k < steps; ++k) {
      // P = X X^T from X^T's columns against themselves; P and Q are their own transposes
      int status = dgemm_region_tn(region, r, r, c, XT, c, XT, c, P, r, s, st);
      if (!status) status = dgemm_region_tn(region, r, r, r, P, r, P, r, Q, r, s, st);
      if (status) return status;
      const long rr = (long)r * r;
      hipLaunchKernelGGL(combine64_kernel, dim3((unsigned)((rr + 255) / 256)), dim3(256), 0, st, Q, P, co[3 * k + 1],
                         co[3 * k + 2], rr);
      if ((status = dgemm_region_tn(region, r, c, r, Q, r, X, r, Y, r, s, st))) return status;
      hipLaunchKernelGGL(update64_kernel, xt, dim3(256), 0, st, X, XT, Y, co[3 * k], c, r,
                         k + 1 == steps ? Oi : nullptr, ldo, as_it_lies ? 0 : 1);
      OZ_TRY(hipGetLastError());
    }
  }
  return OZGEMM_OK;
}

// The same by the FP64 matrix cores, the whole batch at once.  X stays as G
// lies: n rows of m entries.
int ortho64_direct(const OrthoLayout& L, int batch, int m, int n, const double* G, long ldg, long strideg, int steps,
                   const double* co, double eps, double* O, long ldo, long strideo, char* ws, hipStream_t st) {
  const bool tall = n > m;
  const int r = tall ? m : n, c = tall ? n : m;
  double* X = (double*)(ws + L.X);
  double* other = (double*)(ws + L.Y);
  double* P = (double*)(ws + L.P);
  double* Q = (double*)(ws + L.Q);
  double* part = (double*)(ws + L.part);
  const int parts = square_parts(m, n);
  const long xs = (long)m * n, ps = (long)r * r;
  OZ_TRY(launch_square_sum(OZGEMM_F64, G, n, m, ldg, strideg, batch, parts, part, st));
  hipLaunchKernelGGL(scale64_kernel, dim3((unsigned)((xs + 255) / 256), batch), dim3(256), 0, st, G, n, m, ldg, strideg,
                     part, parts, eps, X);
  OZ_TRY(hipGetLastError());
  // X(r-index i, c-index k) at i x_r + k x_c
  const long x_r = tall ? 1 : m, x_c = tall ? m : 1;
  int units = 0;
  OZ_TRY(device_units(&units));
  auto launch = [&](const Step64& p, bool sym) { return launch_step64(p, sym, units, st); };
  for (int k = 0; k < steps; ++k) {
    const double a = co[3 * k], b = co[3 * k + 1], cc = co[3 * k + 2];
    Step64 p{};
    p.batch = batch;
    p.A = p.B = X;  // P = X X^T
    p.a_i = p.b_j = x_r;
    p.a_k = p.b_k = x_c;
    p.a_batch = p.b_batch = xs;
    p.m = p.n = r;
    p.k = c;
    p.alpha = 1;
    p.N = P;
    p.n_ld = r;
    p.n_batch = ps;
    OZ_TRY(launch(p, true));
    p.A = p.B = P;  // Q = b P + c P^2
    p.a_i = p.b_j = r;
    p.a_k = p.b_k = 1;
    p.a_batch = p.b_batch = ps;
    p.k = r;
    p.alpha = cc;
    p.beta = b;
    p.S = P;
    p.s_ld = r;
    p.s_batch = ps;
    p.N = Q;
    OZ_TRY(launch(p, true));
    // X <- a X + Q X, row j of the result as X lies: wide, row j of Q against
    // X's columns; tall, row j of X against Q
    p.A = tall ? Q : X;
    p.a_i = tall ? r : x_c;
    p.a_k = tall ? 1 : x_r;
    p.a_batch = tall ? ps : xs;
    p.B = tall ? X : Q;
    p.b_j = tall ? x_c : r;
    p.b_k = 1;
    p.b_batch = tall ? xs : ps;
    p.m = m;
    p.n = n;
    p.k = r;
    p.alpha = 1;
    p.beta = a;
    p.S = X;
    p.s_ld = m;
    p.s_batch = xs;
    const bool last = k + 1 == steps;
    p.N = last ? O : other;
    p.n_ld = last ? ldo : m;
    p.n_batch = last ? strideo : xs;
    OZ_TRY(launch(p, false));
    double* swap = X;
    X = other;
    other = swap;
  }
  return OZGEMM_OK;
}

int ortho16(const OrthoLayout& L, int type, int batch, int m, int n, const void* G, long ldg, long strideg, int steps,
            const double* co, double eps, void* O, long ldo, long strideo, char* ws, hipStream_t st) {
  const bool tall = n > m;  // as it lies: n rows of m entries
  uint16_t* X = (uint16_t*)(ws + L.X1);
  uint16_t* other = (uint16_t*)(ws + L.X2);
  uint16_t* P = (uint16_t*)(ws + L.P);
  uint16_t* Q = (uint16_t*)(ws + L.Q);
  double* part = (double*)(ws + L.part);
  const long xp = (long)L.rp * L.cp, pp = (long)L.rp * L.rp;
  const int parts = square_parts(m, n);
  StepFactors* factors = (StepFactors*)(ws + L.factors);
  OZ_TRY(launch_square_sum(type, G, n, m, ldg, strideg, batch, parts, part, st));
  Prepare pr{G, n, m, ldg, strideg, part, parts, eps, X, tall ? L.cp : L.rp, tall ? L.rp : L.cp,
             xp / 8 * batch < 4096L * 256 ? 1 : PREPARE_RUNS, factors, steps, batch, {}};
  for (int i = 0; i < 3 * steps; ++i) pr.co[i] = co[i];
  const dim3 blocks((unsigned)((xp / 8 + 256 * pr.each - 1) / (256 * pr.each)) + 1, batch);
  if (type == OZGEMM_F32)
    hipLaunchKernelGGL(prepare_kernel<OZGEMM_F32>, blocks, dim3(256), 0, st, pr);
  else if (type == OZGEMM_BF16)
    hipLaunchKernelGGL(prepare_kernel<OZGEMM_BF16>, blocks, dim3(256), 0, st, pr);
  else
    hipLaunchKernelGGL(prepare_kernel<OZGEMM_F16>, blocks, dim3(256), 0, st, pr);
  OZ_TRY(hipGetLastError());
  for (int k = 0; k < steps; ++k) {
    const int x_ld = tall ? L.rp : L.cp;
    Step p{};
    p.batch = batch;
    p.factors = factors + (long)k * batch;
    // P = X X^T along the c entries: next to each other in a wide X, a row apart in a tall one
    p.A = p.B = X;
    p.a_batch = p.b_batch = 2 * xp;
    p.a_plane = p.b_plane = xp;
    p.a_ld = p.b_ld = x_ld;
    p.m = p.n = L.rp;
    p.k = L.cp;
    p.which = 0;
    p.N = P;
    p.s_batch = 2 * pp;
    p.s_plane = pp;
    if (L.parts > 1)
      OZ_TRY(launch_gram_parts(Parts{X, 2 * xp, xp, x_ld, L.rp, L.cp, batch, L.parts, p.factors,
                                     (float*)(ws + L.partial), P}, tall, st));
    else
      OZ_TRY(launch_step(p, tall, true, st));
    // Q = b P + c P^2
    p.A = p.B = P;
    p.a_batch = p.b_batch = 2 * pp;
    p.a_plane = p.b_plane = pp;
    p.a_ld = p.b_ld = L.rp;
    p.k = L.rp;
    p.which = 1;
    p.S = P;
    p.N = Q;
    OZ_TRY(launch_step(p, false, true, st));
    // X <- a X + Q X along the r rows, the result as X lies: wide, its row j
    // is row j of Q against X's columns; tall, row j of X against Q
    p.A = tall ? Q : X;
    p.B = tall ? X : Q;
    p.a_batch = tall ? 2 * pp : 2 * xp;
    p.a_plane = tall ? pp : xp;
    p.a_ld = tall ? L.rp : x_ld;
    p.b_batch = tall ? 2 * xp : 2 * pp;
    p.b_plane = tall ? xp : pp;
    p.b_ld = tall ? x_ld : L.rp;
    p.m = tall ? L.rp : L.cp;
    p.n = tall ? L.cp : L.rp;
    p.which = 2;
    p.S = X;
    p.N = other;
    p.s_batch = 2 * xp;
    p.s_plane = xp;
    if (k + 1 == steps) {
      p.O = O;
      p.otype = type;
      p.ldo = ldo;
      p.batcho = strideo;
      p.om = m;
      p.on = n;
    }
    OZ_TRY(launch_step(p, !tall, false, st));
    uint16_t* swap = X;
    X = other;
    other = swap;
  }
  return OZGEMM_OK;
}

size_t span(int m, int n, long ld, long long stride, int batch, size_t size) {
  if (m < 1 || n < 1 || batch < 1) return 0;
  return ((size_t)(batch - 1) * (size_t)stride + (size_t)(n - 1) * (size_t)ld + (size_t)m) * size;
}

bool ortho_range(int type, int batch, int m, int n, int s) {
  if (m > OZGEMM_ORTHO_MAX || n > OZGEMM_ORTHO_MAX || batch > 65535) return false;
  return type != OZGEMM_F64 || (ozgemm_kbits(s, m > n ? m : n) >= 1);
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozgemm_orthogonalize_workspace_bytes(int type, int batch, int m, int n, int s) {
  if (type < OZGEMM_F64 || type > OZGEMM_F16 || batch < 1 || m < 1 || n < 1) return 0;
  if (type == OZGEMM_F64 && (s < 1 || s > OZGEMM_S_MAX)) return 0;
  if (!ortho_range(type, batch, m, n, s)) return 0;
  return ortho_layout(type, batch, m, n, s).total;
}

int ozgemm_orthogonalize(int type, int batch, int m, int n, const void* G, int ldg, long long strideg, int steps,
                         const double* coeffs, double eps, int s, void* O, int ldo, long long strideo,
                         void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (type < OZGEMM_F64 || type > OZGEMM_F16) return -1;
  if (batch < 0) return -2;
  if (m < 0) return -3;
  if (n < 0) return -4;
  const bool any = batch > 0 && m > 0 && n > 0;
  if (G == nullptr && any) return -5;
  if (ldg < (m > 1 ? m : 1)) return -6;
  if (strideg < 0) return -7;
  if (steps < 0 || steps > OZGEMM_ORTHO_STEPS_MAX) return -8;
  if (coeffs == nullptr && steps > 0) return -9;
  for (int i = 0; i < 3 * steps; ++i)
    if (!(fabs(coeffs[i]) < 1e6)) return -9;
  if (!(eps >= 0) || !(eps < 1e300)) return -10;
  if (type == OZGEMM_F64 && (s < 1 || s > OZGEMM_S_MAX)) return -11;
  if (O == nullptr && any) return -12;
  if (ldo < (m > 1 ? m : 1)) return -13;
  if (strideo < 0 || (any && batch > 1 && strideo < (long long)ldo * (n - 1) + m)) return -14;
  if (any && !ortho_range(type, batch, m, n, s)) return OZGEMM_RANGE;
  const size_t size = elem_bytes(type);
  if (any && !(O == G && ldo == ldg && (batch == 1 || strideo == strideg))) {
    const char* o = (const char*)O;
    const char* gg = (const char*)G;
    if (o < gg + span(m, n, ldg, strideg, batch, size) && gg < o + span(m, n, ldo, strideo, batch, size)) return -12;
  }
  if (any && (workspace == nullptr || ((uintptr_t)workspace & 255))) return -15;
  if (!any) return OZGEMM_OK;
  if (type != OZGEMM_F64 && !schedule_fits(coeffs, steps)) return OZGEMM_RANGE;
  const OrthoLayout L = ortho_layout(type, batch, m, n, s);
  if (workspace_bytes < L.total) return OZGEMM_WORKSPACE_TOO_SMALL;
  hipStream_t st = (hipStream_t)hip_stream;
  char* ws = (char*)workspace;
  if (steps == 0) {
    const int parts = square_parts(m, n);
    double* part = (double*)(ws + L.part);
    OZ_TRY(launch_square_sum(type, G, n, m, ldg, (long)strideg, batch, parts, part, st));
    const long total = (long)m * n;
    in_pieces((total + 255) / 256, [&](long first, unsigned count) {
      hipLaunchKernelGGL(normalise_kernel, dim3(count, batch), dim3(256), 0, st, G, type, n, m, (long)ldg,
                         (long)strideg, part, parts, eps, O, (long)ldo, (long)strideo, first);
    });
    OZ_TRY(hipGetLastError());
    return OZGEMM_OK;
  }
  if (type == OZGEMM_F64 && L.direct)
    return ortho64_direct(L, batch, m, n, (const double*)G, ldg, (long)strideg, steps, coeffs, eps, (double*)O, ldo,
                          (long)strideo, ws, st);
  if (type == OZGEMM_F64)
    return ortho64(L, batch, m, n, (const double*)G, ldg, (long)strideg, steps, coeffs, eps, s, (double*)O, ldo,
                   (long)strideo, ws, st);
  return ortho16(L, type, batch, m, n, G, ldg, (long)strideg, steps, coeffs, eps, O, ldo, (long)strideo, ws, st);
}

}  // extern "C"
