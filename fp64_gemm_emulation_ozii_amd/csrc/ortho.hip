// Orthogonalisation by Newton-Schulz products:
//   X_0 = G / (|G|_F + eps),  P = X X^T,  Q = b P + c P^2,  X <- a X + Q X,
// X with its r rows no more than its c columns (G or its transpose; the
// iteration commutes with the transpose).
//
// Everything between G and the result stays in half-precision slices
// (slices.hip): x S = hi + lo with a power of two S that the host derives
// from a bound on the iterate's singular values, which keeps 22 bits or more
// of every state whatever the type.  BF16 operands use one slice product
// (hi hi: its operands are off by 2^-11, an eighth of the result's own
// rounding; the term a X, through which small singular values grow 3.4 times
// a step, uses both slices, so rounding is not amplified with them).  F16 and
// F32 use three.  F64 runs the library's Scheme II products.
//
// X is kept both ways round (Xr: r x c, Xc: c x r), so that every product
// has both operands K-contiguous; the step that writes X writes both.  P
// and P^2 are symmetric: tiles on and below the diagonal are computed and
// written twice.
#include <hip/hip_runtime.h>

#include <cmath>

#include "products.h"
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

// Sums of squares in FP64 (no square of an FP32 value leaves its range):
// block (p, b) adds its share of the rows of matrix b.
__global__ __launch_bounds__(256) void square_sum_kernel(const void* __restrict__ G, int type, int rows, int cols,
                                                         long ld, long batch, double* __restrict__ part) {
  __shared__ double s[4];
  const long base = blockIdx.y * batch;
  double sum = 0;
  const long total = (long)rows * cols;
  for (long at = (long)blockIdx.x * 256 + threadIdx.x; at < total; at += (long)gridDim.x * 256) {
    const long r = at / cols;
    const double v = load_value(G, type, base + r * ld + (at - r * cols));
    sum += v * v;
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// 1 / (|G_b|_F + eps) from the partial sums of matrix b, in every thread of the block.
__device__ __forceinline__ double inverse_norm(const double* part, int parts, long b, double eps, double* s) {
  const double v = block_sum((int)threadIdx.x < parts ? part[b * parts + threadIdx.x] : 0.0, s);
  return 1.0 / (sqrt(v) + eps);
}

__device__ __forceinline__ void split(float y, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)y;
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, (_Float16)(y - (float)h));
}

__device__ __forceinline__ float joined(uint16_t hi, uint16_t lo) {
  return (float)__builtin_bit_cast(_Float16, hi) + (float)__builtin_bit_cast(_Float16, lo);
}

// G (rows x cols) scaled and cut into slices, as it lies (N: np x kp) and
// transposed (T: kp x np), zeros in the padding.
struct Prepare {
  const void* G;
  int type;
  int rows, cols;
  long ld, batch;
  const double* part;
  int parts;
  double eps, scale;
  uint16_t* N;   // [batch][2][rows_pad][cols_pad]
  uint16_t* T;   // [batch][2][cols_pad][rows_pad]
  int rows_pad, cols_pad;
};

__global__ __launch_bounds__(256) void prepare_kernel(Prepare p) {
  __shared__ double s[4];
  __shared__ uint32_t tile[64][65];
  const long b = blockIdx.z;
  const double f = inverse_norm(p.part, p.parts, b, p.eps, s) * p.scale;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const long plane = (long)p.rows_pad * p.cols_pad;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = r0 + (i >> 6), c = c0 + (i & 63);
    uint16_t hi = 0, lo = 0;
    if (r < p.rows && c < p.cols) split((float)(load_value(p.G, p.type, b * p.batch + r * p.ld + c) * f), hi, lo);
    const long at = b * 2 * plane + (long)r * p.cols_pad + c;
    p.N[at] = hi;
    p.N[at + plane] = lo;
    tile[i >> 6][i & 63] = hi | ((uint32_t)lo << 16);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = i >> 6, r = i & 63;
    const long at = b * 2 * plane + (long)(c0 + c) * p.rows_pad + r0 + r;
    p.T[at] = (uint16_t)tile[r][c];
    p.T[at + plane] = (uint16_t)(tile[r][c] >> 16);
  }
}

__global__ __launch_bounds__(256) void normalise_kernel(const void* G, int type, int rows, int cols, long ld,
                                                        long batch, const double* __restrict__ part, int parts,
                                                        double eps, void* O, long ldo, long batcho) {
  __shared__ double s[4];
  const long b = blockIdx.y;
  const double f = inverse_norm(part, parts, b, eps, s);
  const long at = (long)blockIdx.x * 256 + threadIdx.x;
  if (at >= (long)rows * cols) return;
  const long r = at / cols, c = at - r * cols;
  store_value(O, type, b * batcho + r * ldo + c, load_value(G, type, b * batch + r * ld + c) * f);
}

// One product of a step: D = A B^T on padded planes, then
// v = alpha D + beta S, rounded to slices of N ([j][i]) and of T ([i][j]),
// or, last, to the result.
struct Step {
  const uint16_t* A;  // [batch] a_batch apart, two slices a_plane apart, rows of k entries
  const uint16_t* B;
  long a_batch, a_plane, b_batch, b_plane;
  int m, n, k;        // padded
  int nprod, symmetric;
  float alpha, beta;
  const uint16_t* S;  // like N; nullptr: beta = 0
  uint16_t* N;
  uint16_t* T;
  long s_batch, s_plane;  // of S, N and T alike
  int s_lo, n_lo, t_lo;   // whether the low slices are there
  void* O;
  int otype;
  long ldo, batcho;
  int om, on;         // the result's own size
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void step_kernel(Step p) {
  using Tile = Tile16<Half, BM, BN, WM, WN, false, false>;
  __shared__ __attribute__((aligned(1024))) char smem[Tile::SMEM];
  const int tm = p.m / BM, tn = p.n / BN;
  int mi, nj;
  if (p.symmetric) {  // tiles (mi, nj), nj <= mi, by rows of the triangle
    const int t = blockIdx.x;
    mi = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while ((mi + 1) * (mi + 2) / 2 <= t) ++mi;
    while (mi * (mi + 1) / 2 > t) --mi;
    nj = t - mi * (mi + 1) / 2;
  } else {
    mi = blockIdx.x % tm;
    nj = blockIdx.x / tm;
  }
  (void)tn;
  const long b = blockIdx.y;
  const int m0 = mi * BM, n0 = nj * BN;
  const Source16 A{p.A + b * p.a_batch + (long)m0 * p.k, p.a_plane, p.k, p.m - m0, p.k};
  const Source16 B{p.B + b * p.b_batch + (long)n0 * p.k, p.b_plane, p.k, p.n - n0, p.k};
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, A, B, p.k, p.nprod);

  constexpr int WTM = Tile::FM * 16, PITCH = WTM + 4, RUNS = WTM / 8;
  static_assert(Tile::NW * 16 * PITCH * 4 <= Tile::SMEM, "staging fits the operand buffers");
  slice_barrier();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* stage = reinterpret_cast<float*>(smem) + wave * 16 * PITCH;
  const int mw = m0 + wave / WN * WTM, nw = n0 + wave % WN * (Tile::FN * 16);
  const uint16_t* S = p.S ? p.S + b * p.s_batch : nullptr;
  uint16_t* N = p.N + b * p.s_batch;
  uint16_t* T = p.T + b * p.s_batch;
  const bool mirror = !(p.symmetric && mi == nj);  // a diagonal tile holds both halves itself
#pragma unroll
  for (int j = 0; j < Tile::FN; ++j) {
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
      *reinterpret_cast<v4f*>(stage + (lane & 15) * PITCH + i * 16 + 4 * (lane >> 4)) = acc[i][j];
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
#pragma unroll 1
    for (int at = lane; at < 16 * RUNS; at += 64) {
      const int c = at / RUNS, r = at % RUNS * 8;
      const int col = nw + j * 16 + c, row = mw + r;
      float v[8];
      *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r);
      *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r + 4);
      const long off = (long)col * p.m + row;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= p.alpha;
      if (S != nullptr) {
        const v8s h = *reinterpret_cast<const v8s*>(S + off);
        v8s l = {0, 0, 0, 0, 0, 0, 0, 0};
        if (p.s_lo) l = *reinterpret_cast<const v8s*>(S + p.s_plane + off);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(p.beta, joined((uint16_t)h[e], (uint16_t)l[e]), v[e]);
      }
      if (p.O != nullptr) {
        if (col < p.on) {
          const long to = b * p.batcho + (long)col * p.ldo + row;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row + e < p.om) store_value(p.O, p.otype, to + e, v[e]);
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
      *reinterpret_cast<v8s*>(N + off) = h;
      if (p.n_lo) *reinterpret_cast<v8s*>(N + p.s_plane + off) = l;
      // the rounded slices go back to the staging piece for the transposed copy
      if (mirror) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint32_t*>(stage)[c * PITCH + r + e] = (uint16_t)h[e] | ((uint32_t)(uint16_t)l[e] << 16);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
    if (p.O == nullptr && mirror) {
      // 16 columns of one row: 32 bytes
#pragma unroll 1
      for (int at = lane; at < WTM * 2; at += 64) {
        const int r = at >> 1, c = (at & 1) * 8;
        v8s h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(stage)[(c + e) * PITCH + r];
          h[e] = (short)w;
          l[e] = (short)(w >> 16);
        }
        const long off = (long)(mw + r) * p.n + nw + j * 16 + c;
        *reinterpret_cast<v8s*>(T + off) = h;
        if (p.t_lo) *reinterpret_cast<v8s*>(T + p.s_plane + off) = l;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
      asm volatile("" ::: "memory");
    }
  }
}

template <int BT, int WM, int WN>
hipError_t launch_step_t(const Step& p, int batch, hipStream_t st) {
  const long tm = p.m / BT, tn = p.n / BT;
  const long tiles = p.symmetric ? tm * (tm + 1) / 2 : tm * tn;
  hipLaunchKernelGGL((step_kernel<BT, BT, WM, WN>), dim3((unsigned)tiles, (unsigned)batch), dim3(WM * WN * 64), 0, st,
                     p);
  return hipGetLastError();
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

// Blocks that sum one matrix's squares: 16 entries a thread, SQUARE_PARTS at most.
int square_parts(int m, int n) {
  const long blocks = ((long)m * n + 4095) / 4096;
  return (int)(blocks < 1 ? 1 : blocks > SQUARE_PARTS ? SQUARE_PARTS : blocks);
}

// Tile size of the step products: the padded matrix is cut into whole tiles.
int step_tile(int batch, int r, int c) {
  (void)batch;
  if (r <= 64 || c <= 64) return 64;
  return 128;
}

struct OrthoLayout {
  int tile, rp, cp;
  size_t part, Xr, Xc, Xc2, P, Q, total;   // 16-bit types
  size_t X, XT, Y, dgemm;                  // FP64
};

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
    L.X = take(rc);
    L.XT = take(rc);
    L.Y = take(rc);
    L.P = take(rr);
    L.Q = take(rr);
    L.dgemm = take(dgemm_region_bytes(r, c, s));
    return L;
  }
  L.tile = step_tile(batch, r, c);
  L.rp = (int)up(r, L.tile);
  L.cp = (int)up(c, L.tile);
  const size_t rc = (size_t)batch * 2 * L.rp * L.cp * 2, rr = (size_t)batch * 2 * L.rp * L.rp * 2;
  L.Xr = take(rc);
  L.Xc = take(rc);
  L.Xc2 = take(rc);
  L.P = take(rr);
  L.Q = take(rr);
  return L;
}

// Slice products of a step.  One is enough for BF16 results: at 1024 rows the
// error is 1.2 to 1.35 times the rounding of the result alone.  It falls with
// the smaller side r (1.1 at 2048, 1.6 at 64), and below 256 rows, where a
// call is bound by its launches, three cost little and leave the rounding alone.
int ortho_products(int type, int r) { return type == OZGEMM_BF16 && r >= 256 ? 1 : 3; }

// Largest |p| over [0, t] of p(x) = a x + b x^3 + c x^5: at t or where
// a + 3 b y + 5 c y^2 = 0, y = x^2.
double peak(double a, double b, double c, double t) {
  auto p = [&](double x) { return fabs(x * (a + x * x * (b + x * x * c))); };
  double top = p(t);
  double roots[2] = {-1, -1};
  if (c != 0) {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      roots[0] = (-3 * b + sqrt(d)) / (10 * c);
      roots[1] = (-3 * b - sqrt(d)) / (10 * c);
    }
  } else if (b != 0) {
    roots[0] = -a / (3 * b);
  }
  for (double y : roots)
    if (y > 0 && y < t * t) top = fmax(top, p(sqrt(y)));
  return top;
}

// Largest |b y + c y^2| over [0, u].
double peak_q(double b, double c, double u) {
  double top = fabs(u * (b + c * u));
  if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < u) top = fmax(top, fabs(b * b / (4 * c)));
  return top;
}

// Power of two S with bound S in [2^13, 2^14): an entry may pass the bound four
// times over before it leaves half's range (65504).  The bounds hold for the
// exact iteration; they carry no further margin, because the polynomials of
// a schedule grow steeply past the interval they are made for and every bit
// given away here is lost to the low slices.
bool grid(double bound, double* S) {
  if (!(bound < 1e18)) return false;
  int e = 0;
  frexp(fmax(bound, 1e-6), &e);
  *S = ldexp(1.0, 14 - e);
  return true;
}

#define OZ_TRY(expr)                                                   \
  do {                                                                 \
    const hipError_t oz_err_ = (expr);                                 \
    if (oz_err_ != hipSuccess) return record_hip_error(oz_err_);       \
  } while (0)

struct Scales {
  double X, P, Q, next;
};

// The grids of every step; false where the bound leaves a double's sensible range.
bool scales_of(const double* co, int steps, int i, double* t, Scales* out) {
  (void)steps;
  const double a = co[3 * i], b = co[3 * i + 1], c = co[3 * i + 2];
  const double u = *t * *t;
  const double after = peak(a, b, c, *t) * (1 + 1.0 / 1024);
  if (!grid(*t, &out->X) || !grid(u, &out->P) || !grid(peak_q(b, c, u), &out->Q) || !grid(after, &out->next))
    return false;
  *t = after;
  return true;
}

constexpr double START = 1.0;  // |X_0| <= 1

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
    hipLaunchKernelGGL(square_sum_kernel, dim3(parts, 1), dim3(256), 0, st, Gi, OZGEMM_F64, n, m, ldg, 0L, part);
    hipLaunchKernelGGL(prepare64_kernel, tiles, dim3(256), 0, st, Gi, n, m, ldg, part, parts, eps,
                       as_it_lies ? X : XT, as_it_lies ? XT : X);
    OZ_TRY(hipGetLastError());
    for (int k = 0; k < steps; ++k) {
      int status = dgemm_region(region, r, r, c, X, r, XT, c, P, r, s, st);
      if (!status) status = dgemm_region(region, r, r, r, P, r, P, r, Q, r, s, st);
      if (status) return status;
      const long rr = (long)r * r;
      hipLaunchKernelGGL(combine64_kernel, dim3((unsigned)((rr + 255) / 256)), dim3(256), 0, st, Q, P, co[3 * k + 1],
                         co[3 * k + 2], rr);
      if ((status = dgemm_region(region, r, c, r, Q, r, X, r, Y, r, s, st))) return status;
      hipLaunchKernelGGL(update64_kernel, xt, dim3(256), 0, st, X, XT, Y, co[3 * k], c, r,
                         k + 1 == steps ? Oi : nullptr, ldo, as_it_lies ? 0 : 1);
      OZ_TRY(hipGetLastError());
    }
  }
  return OZGEMM_OK;
}

int ortho16(const OrthoLayout& L, int type, int batch, int m, int n, const void* G, long ldg, long strideg, int steps,
            const double* co, double eps, void* O, long ldo, long strideo, char* ws, hipStream_t st) {
  const bool tall = n > m;  // as it lies: n rows of m entries
  const int r = tall ? m : n;
  uint16_t* Xr = (uint16_t*)(ws + L.Xr);
  uint16_t* Xc = (uint16_t*)(ws + L.Xc);
  uint16_t* Xc2 = (uint16_t*)(ws + L.Xc2);
  uint16_t* P = (uint16_t*)(ws + L.P);
  uint16_t* Q = (uint16_t*)(ws + L.Q);
  double* part = (double*)(ws + L.part);
  const long xp = (long)L.rp * L.cp, pp = (long)L.rp * L.rp;
  const int nprod = ortho_products(type, r), lo = nprod == 3;
  const int parts = square_parts(m, n);
  double t = START;
  Scales sc;
  if (!scales_of(co, steps, 0, &t, &sc)) return OZGEMM_RANGE;
  hipLaunchKernelGGL(square_sum_kernel, dim3(parts, batch), dim3(256), 0, st, G, type, n, m, ldg, strideg, part);
  Prepare pr{G, type, n, m, ldg, strideg, part, parts, eps, sc.X, tall ? Xc : Xr, tall ? Xr : Xc,
             tall ? L.cp : L.rp, tall ? L.rp : L.cp};
  hipLaunchKernelGGL(prepare_kernel, dim3(pr.cols_pad / 64, pr.rows_pad / 64, batch), dim3(256), 0, st, pr);
  OZ_TRY(hipGetLastError());
  auto launch = [&](const Step& p) {
    return L.tile == 64 ? launch_step_t<64, 2, 2>(p, batch, st) : launch_step_t<128, 2, 2>(p, batch, st);
  };
  t = START;
  for (int k = 0; k < steps; ++k) {
    if (!scales_of(co, steps, k, &t, &sc)) return OZGEMM_RANGE;
    const double a = co[3 * k], b = co[3 * k + 1], c = co[3 * k + 2];
    Step p{};
    p.nprod = nprod;
    // P = X X^T
    p.A = p.B = Xr;
    p.a_batch = p.b_batch = 2 * xp;
    p.a_plane = p.b_plane = xp;
    p.m = p.n = L.rp;
    p.k = L.cp;
    p.symmetric = 1;
    p.alpha = (float)(sc.P / (sc.X * sc.X));
    p.N = p.T = P;
    p.s_batch = 2 * pp;
    p.s_plane = pp;
    p.n_lo = p.t_lo = lo;
    OZ_TRY(launch(p));
    // Q = b P + c P^2
    p.A = p.B = P;
    p.a_batch = p.b_batch = 2 * pp;
    p.a_plane = p.b_plane = pp;
    p.k = L.rp;
    p.alpha = (float)(c * sc.Q / (sc.P * sc.P));
    p.beta = (float)(b * sc.Q / sc.P);
    p.S = P;
    p.s_lo = lo;
    p.N = p.T = Q;
    OZ_TRY(launch(p));
    // X <- a X + Q X: tall results lie c x r (rows of X^T against Q), wide ones r x c
    p.A = tall ? Q : Xc;
    p.B = tall ? Xc : Q;
    p.a_batch = tall ? 2 * pp : 2 * xp;
    p.a_plane = tall ? pp : xp;
    p.b_batch = tall ? 2 * xp : 2 * pp;
    p.b_plane = tall ? xp : pp;
    p.m = tall ? L.rp : L.cp;
    p.n = tall ? L.cp : L.rp;
    p.symmetric = 0;
    const double next = k + 1 < steps ? sc.next : 1.0;  // the result itself is on no grid
    p.alpha = (float)(next / (sc.Q * sc.X));
    p.beta = (float)(a * next / sc.X);
    p.S = tall ? Xc : Xr;
    p.s_lo = 1;
    p.N = tall ? Xc2 : Xr;
    p.T = tall ? Xr : Xc2;
    p.s_batch = 2 * xp;
    p.s_plane = xp;
    p.n_lo = 1;
    p.t_lo = lo;
    if (k + 1 == steps) {
      p.O = O;
      p.otype = type;
      p.ldo = ldo;
      p.batcho = strideo;
      p.om = m;
      p.on = n;
    }
    OZ_TRY(launch(p));
    uint16_t* swap = Xc;
    Xc = Xc2;
    Xc2 = swap;
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
  double t = START;
  Scales sc;
  if (type != OZGEMM_F64)
    for (int k = 0; k < steps; ++k)
      if (!scales_of(coeffs, steps, k, &t, &sc)) return OZGEMM_RANGE;
  const OrthoLayout L = ortho_layout(type, batch, m, n, s);
  if (workspace_bytes < L.total) return OZGEMM_WORKSPACE_TOO_SMALL;
  hipStream_t st = (hipStream_t)hip_stream;
  char* ws = (char*)workspace;
  if (steps == 0) {
    const int parts = square_parts(m, n);
    double* part = (double*)(ws + L.part);
    hipLaunchKernelGGL(square_sum_kernel, dim3(parts, batch), dim3(256), 0, st, G, type, n, m, (long)ldg,
                       (long)strideg, part);
    const long total = (long)m * n;
    hipLaunchKernelGGL(normalise_kernel, dim3((unsigned)((total + 255) / 256), batch), dim3(256), 0, st, G, type, n, m,
                       (long)ldg, (long)strideg, part, parts, eps, O, (long)ldo, (long)strideo);
    OZ_TRY(hipGetLastError());
    return OZGEMM_OK;
  }
  if (type == OZGEMM_F64)
    return ortho64(L, batch, m, n, (const double*)G, ldg, (long)strideg, steps, coeffs, eps, s, (double*)O, ldo,
                   (long)strideo, ws, st);
  return ortho16(L, type, batch, m, n, G, ldg, (long)strideg, steps, coeffs, eps, O, ldo, (long)strideo, ws, st);
}

}  // extern "C"
