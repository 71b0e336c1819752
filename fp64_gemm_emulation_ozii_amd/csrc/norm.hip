// Root-mean-square norm of rows, with the residual's addition before it and
// values in 8 bits behind it, and its gradients.
//
//   H = X + R (each entry rounded to their type),  r = 1 / sqrt(sum H^2 / q + eps),  Y = H r w
//   g = dY w,  dX = r g - H r^3 (sum g H) / q + dH,  dw = sum over the rows of dY H r
// The middle term is formed as (H r) (r^2 sum g H / q): with a third r in its second factor that would leave
// float32's range for rows below 1e-19 (where eps is 0).  r itself leaves it below 3e-39.
//
// G threads hold a row of up to 8192 entries in registers, eight entries P times
// each, so it is read once.  Sums over a row and Y itself are FP64: that costs nothing next to the
// memory, and every value of Y, its block's scale and its 8 bits are the
// rounded exact ones (to_odd, block8.h) instead of ones that flip where an
// FP32 value lies next to a border.
//
// Bound by HBM: 8192 x 4096 of BF16 with a residual, to 8 bits, 45 us or 5.2 TB/s;
// 16384 x 2048, with a residual, 58 us or 4.6 TB/s; its gradients 55 us or 4.9 TB/s
// and 4 us for the sums of dw (a large copy: 4.9).  One row of 4096: 3.7 us.
#include <algorithm>

#include "block8.h"
#include "products.h"

namespace oz {
namespace {

struct Norm {
  const void *x, *res, *w;
  void *h, *y;
  float* s;
  long ldx, ldres, ldh, ldy, srow, sblock;
  int n, q, wf32;
  double eps;
};

template <int G>
__device__ __forceinline__ double row_sum(double v, double* meet) {
  v = sum64(v);
  if (G > 64) {
    __syncthreads();  // (the row before has been read)
    if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = v;
    __syncthreads();
    v = meet[0];
#pragma unroll
    for (int k = 1; k < G / 64; ++k) v += meet[k];
  }
  return v;
}

template <int TYPE>
__device__ __forceinline__ void load_weights(float (&w)[8], const void* from, int wf32, int c, int q) {
  if (c >= q) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 0.f;
  } else if (wf32) {
    Raw8<OZGEMM_F32> v;
    v.load(from, c, q - c);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = v.get(k);
  } else {
    Raw8<TYPE> v;
    v.load(from, c, q - c);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = v.get(k);
  }
}

// Eight entries of Y; OUT: its type, TYPE or an 8-bit one, whose blocks are 16
// neighbouring lanes' (all of which come here).
template <int TYPE, int OUT>
__device__ __forceinline__ void store_y(const Norm& g, long row, int c, int t, const Raw8<TYPE>& h, double r,
                                        const float (&w)[8]) {
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const double v = (double)h.get(k) * r * (double)w[k];
    y[k] = OUT == OZGEMM_F32 ? (float)v : to_odd(v);  // (rounded again below where it is shorter)
  }
  if constexpr (OUT == OZGEMM_E4M3 || OUT == OZGEMM_E5M2) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, finite_abs(y[k]));
    const int e = scale_exponent<OUT>(max16(m));
    if (c < g.q) {
      const float f = power_of_two(-e);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = no_inf(y[k]) * f;
      store_bytes((uint8_t*)g.y + row * g.ldy + c,
                  v2u{Eight<OUT>::pack4(y[0], y[1], y[2], y[3]), Eight<OUT>::pack4(y[4], y[5], y[6], y[7])}, g.q - c);
      if ((t & 15) == 0) g.s[row * g.srow + c / BLOCK8 * g.sblock] = power_of_two(e);
    }
  } else if (c < g.q) {
    Raw8<TYPE> o;
    o.set(y);
    o.store(g.y, row * g.ldy + c, g.q - c);
  }
}

template <int TYPE, int OUT, int G, int P>
__global__ __launch_bounds__(256) void norm_kernel(Norm g) {
  constexpr int RB = 256 / G;
  __shared__ double meet[G / 64 + 1];
  const int t = threadIdx.x % G;
  float w[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) load_weights<TYPE>(w[p], g.w, g.wf32, (p * G + t) * 8, g.q);
  for (long row = (long)blockIdx.x * RB + threadIdx.x / G; row < g.n; row += (long)gridDim.x * RB) {
    Raw8<TYPE> h[P], res[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t) * 8;
      if (c < g.q) {
        h[p].load(g.x, row * g.ldx + c, g.q - c);
        if (g.res != nullptr) res[p].load(g.res, row * g.ldres + c, g.q - c);
      } else {
        h[p].zero();
        res[p].zero();
      }
    }
    if (g.res != nullptr) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = h[p].get(k) + res[p].get(k);
        h[p].set(v);
        const int c = (p * G + t) * 8;
        if (c < g.q) h[p].store(g.h, row * g.ldh + c, g.q - c);
      }
    }
    double sum = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double v = (double)h[p].get(k);
        sum = __builtin_fma(v, v, sum);
      }
    sum = row_sum<G>(sum, meet);
    const double r = 1.0 / sqrt(sum / (double)g.q + g.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t) * 8;
      store_y<TYPE, OUT>(g, row, c, t, h[p], r, w[p]);
    }
  }
}

// Rows that no block holds: read twice, the second time from H or X and mostly from the caches.
constexpr int LONG = 1024;
template <int TYPE, int OUT>
__global__ __launch_bounds__(LONG) void norm_long_kernel(Norm g) {
  __shared__ double meet[LONG / 64];
  const int t = threadIdx.x;
  const long row = blockIdx.x;
  double sum = 0;
  for (int c = t * 8; c < g.q; c += LONG * 8) {
    Raw8<TYPE> h;
    h.load(g.x, row * g.ldx + c, g.q - c);
    if (g.res != nullptr) {
      Raw8<TYPE> res;
      res.load(g.res, row * g.ldres + c, g.q - c);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = h.get(k) + res.get(k);
      h.set(v);
      h.store(g.h, row * g.ldh + c, g.q - c);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double v = (double)h.get(k);
      sum = __builtin_fma(v, v, sum);
    }
  }
  sum = row_sum<LONG>(sum, meet);
  const double r = 1.0 / sqrt(sum / (double)g.q + g.eps);
  // whole blocks of 16 lanes stay together; each thread reads what it wrote itself
  for (int c = t * 8; c < (g.q + BLOCK8 - 1) / BLOCK8 * BLOCK8; c += LONG * 8) {
    Raw8<TYPE> h;
    if (c >= g.q)
      h.zero();
    else if (g.res != nullptr)
      h.load(g.h, row * g.ldh + c, g.q - c);
    else
      h.load(g.x, row * g.ldx + c, g.q - c);
    float w[8];
    load_weights<TYPE>(w, g.w, g.wf32, c, g.q);
    store_y<TYPE, OUT>(g, row, c, t, h, r, w);
  }
}

struct NormGrads {
  const void *dy, *h, *w, *dh;
  void* dx;
  float* partial;  // [groups][q]; nullptr: no dw
  float* rows;     // long rows: [n][2], r and r^2 (sum g H) / q
  long lddy, ldh, lddh, lddx;
  int n, q, wf32;
  double eps;
};

// Every group of G threads walks its rows and keeps their share of dw in
// registers; a block's groups meet in LDS, and join_weights adds the blocks' in a
// fixed order.
template <int TYPE, int G, int P>
__global__ __launch_bounds__(256) void norm_grads_kernel(NormGrads g) {
  constexpr int RB = 256 / G;
  __shared__ double meet[G / 64 + 1], meet2[G / 64 + 1];
  const int t = threadIdx.x % G;
  float w[P][8], dw[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) load_weights<TYPE>(w[p], g.w, g.wf32, (p * G + t) * 8, g.q);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[p][k] = 0.f;
  for (long row = (long)blockIdx.x * RB + threadIdx.x / G; row < g.n; row += (long)gridDim.x * RB) {
    Raw8<TYPE> h[P], dy[P], dh[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t) * 8;
      if (c < g.q) {
        h[p].load(g.h, row * g.ldh + c, g.q - c);
        dy[p].load(g.dy, row * g.lddy + c, g.q - c);
        if (g.dh != nullptr) dh[p].load(g.dh, row * g.lddh + c, g.q - c);
      } else {
        h[p].zero();
        dy[p].zero();
        dh[p].zero();
      }
    }
    double s1 = 0, s2 = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double v = (double)h[p].get(k);
        s1 = __builtin_fma(v, v, s1);
        s2 = __builtin_fma((double)dy[p].get(k) * (double)w[p][k], v, s2);
      }
    s1 = row_sum<G>(s1, meet);
    s2 = row_sum<G>(s2, meet2);
    const double r = 1.0 / sqrt(s1 / (double)g.q + g.eps);
    const float a = (float)r, b = (float)(r * r * (s2 / (double)g.q));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t) * 8;
      if (c >= g.q) continue;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float hk = a * h[p].get(k), dk = dy[p].get(k);
        v[k] = a * (dk * w[p][k]) - b * hk;
        if (g.dh != nullptr) v[k] += dh[p].get(k);
        dw[p][k] = __builtin_fmaf(dk, hk, dw[p][k]);
      }
      Raw8<TYPE> o;
      o.set(v);
      o.store(g.dx, row * g.lddx + c, g.q - c);
    }
  }
  if (g.partial == nullptr) return;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (p * G + t) * 8;
    if constexpr (RB > 1) {
      __shared__ v4f8 sums[RB - 1][G][2];
      const int group = threadIdx.x / G;
      __syncthreads();  // (the piece before has been read)
      if (group > 0) {
        sums[group - 1][t][0] = v4f8{dw[p][0], dw[p][1], dw[p][2], dw[p][3]};
        sums[group - 1][t][1] = v4f8{dw[p][4], dw[p][5], dw[p][6], dw[p][7]};
      }
      __syncthreads();
      if (group > 0) continue;
#pragma unroll
      for (int o = 0; o < RB - 1; ++o)
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[p][k] += sums[o][t][k >> 2][k & 3];
    }
    Raw8<OZGEMM_F32> o;
    o.set(dw[p]);
    if (c < g.q) o.store(g.partial, (long)blockIdx.x * g.q + c, g.q - c);
  }
}

// Long rows: first what every row needs, then tiles of 2048 columns, whose
// blocks walk every gridDim.y-th row.
template <int TYPE>
__global__ __launch_bounds__(LONG) void norm_grads_rows_kernel(NormGrads g) {
  __shared__ double meet[LONG / 64], meet2[LONG / 64];
  const long row = blockIdx.x;
  double s1 = 0, s2 = 0;
  for (int c = threadIdx.x * 8; c < g.q; c += LONG * 8) {
    Raw8<TYPE> h, dy;
    float w[8];
    h.load(g.h, row * g.ldh + c, g.q - c);
    dy.load(g.dy, row * g.lddy + c, g.q - c);
    load_weights<TYPE>(w, g.w, g.wf32, c, g.q);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double v = (double)h.get(k);
      s1 = __builtin_fma(v, v, s1);
      s2 = __builtin_fma((double)dy.get(k) * (double)w[k], v, s2);
    }
  }
  s1 = row_sum<LONG>(s1, meet);
  s2 = row_sum<LONG>(s2, meet2);
  const double r = 1.0 / sqrt(s1 / (double)g.q + g.eps);
  if (threadIdx.x == 0) {
    g.rows[2 * row] = (float)r;
    g.rows[2 * row + 1] = (float)(r * r * (s2 / (double)g.q));
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void norm_grads_columns_kernel(NormGrads g) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= g.q) return;
  float w[8], dw[8] = {};
  load_weights<TYPE>(w, g.w, g.wf32, c, g.q);
#pragma unroll 2
  for (long row = blockIdx.y; row < g.n; row += gridDim.y) {
    const float a = g.rows[2 * row], b = g.rows[2 * row + 1];
    Raw8<TYPE> h, dy, dh;
    h.load(g.h, row * g.ldh + c, g.q - c);
    dy.load(g.dy, row * g.lddy + c, g.q - c);
    if (g.dh != nullptr) dh.load(g.dh, row * g.lddh + c, g.q - c);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float hk = a * h.get(k), dk = dy.get(k);
      v[k] = a * (dk * w[k]) - b * hk;
      if (g.dh != nullptr) v[k] += dh.get(k);
      dw[k] = __builtin_fmaf(dk, hk, dw[k]);
    }
    Raw8<TYPE> o;
    o.set(v);
    o.store(g.dx, row * g.lddx + c, g.q - c);
  }
  if (g.partial == nullptr) return;
  Raw8<OZGEMM_F32> o;
  o.set(dw);
  o.store(g.partial, (long)blockIdx.y * g.q + c, g.q - c);
}

// dw = the blocks' sums added in FP64: 32 half-wavefronts take every 32nd
// block's, 32 columns each.
__global__ __launch_bounds__(1024) void join_weights_kernel(const float* partial, int groups, int q, void* dw, int type) {
  __shared__ double part[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  double v = 0;
  if (c < q) {
#pragma unroll 8
    for (int i = y; i < groups; i += 32) v += (double)partial[(long)i * q + c];
  }
  part[y][x] = v;
  __syncthreads();
  if (y > 0 || c >= q) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) v += part[k][x];
  const float f = to_odd(v);
  if (type == OZGEMM_F32)
    ((float*)dw)[c] = (float)v;
  else if (type == OZGEMM_BF16)
    ((__bf16*)dw)[c] = (__bf16)f;
  else
    ((_Float16*)dw)[c] = (_Float16)f;
}

// Threads of a row, and how often eight entries each: the first pair that
// holds q ({0, 0}: long rows).
struct Shape {
  int G, P;
};
constexpr Shape SHAPES[] = {{64, 1}, {64, 2}, {256, 1}, {256, 2}, {256, 4}};

Shape shape_of(int q) {
  for (const Shape& s : SHAPES)
    if (q <= s.G * s.P * 8) return s;
  return {0, 0};
}

// call.run<G, P>() with q's shape; whether it has one
template <class Call>
bool with_shape(int q, const Call& call) {
  const Shape s = shape_of(q);
  if (s.G == 64 && s.P == 1) call.template run<64, 1>();
  if (s.G == 64 && s.P == 2) call.template run<64, 2>();
  if (s.G == 256 && s.P == 1) call.template run<256, 1>();
  if (s.G == 256 && s.P == 2) call.template run<256, 2>();
  if (s.G == 256 && s.P == 4) call.template run<256, 4>();
  return s.G > 0;
}

// Blocks of 256 threads for n rows, which walk them: eight for each of the card's 256 compute units,
// or (gradients, which have a row of dw to hand on each) four.
long blocks_for(int n, int G, int each) { return std::min(((long)n * G + 255) / 256, 256L * each); }

template <int TYPE, int OUT>
struct Forward {
  Norm g;
  hipStream_t st;
  template <int G, int P>
  void run() const {
    norm_kernel<TYPE, OUT, G, P><<<(unsigned)blocks_for(g.n, G, 8), 256, 0, st>>>(g);
  }
};

template <int TYPE, int OUT>
void forward(const Norm& g, hipStream_t st) {
  if (!with_shape(g.q, Forward<TYPE, OUT>{g, st})) norm_long_kernel<TYPE, OUT><<<(unsigned)g.n, LONG, 0, st>>>(g);
}

template <int TYPE>
void forward_type(int ytype, const Norm& g, hipStream_t st) {
  if (ytype == OZGEMM_E4M3)
    forward<TYPE, OZGEMM_E4M3>(g, st);
  else if (ytype == OZGEMM_E5M2)
    forward<TYPE, OZGEMM_E5M2>(g, st);
  else
    forward<TYPE, TYPE>(g, st);
}

// Rows of the partial sums of dw: the blocks of a launch (long rows: its gridDim.y).
int grads_groups(int n, int q) {
  const Shape s = shape_of(q);
  if (s.G == 0) return (int)std::min<long>(n, std::max<long>(1, 2048 / ((q + 2047) / 2048)));
  return (int)blocks_for(n, s.G, 4);
}

size_t grads_partial_bytes(int n, int q) { return up((size_t)grads_groups(n, q) * (size_t)q * sizeof(float), 256); }

size_t grads_workspace(int n, int q, bool dw) {
  return (dw ? grads_partial_bytes(n, q) : 0) + (shape_of(q).G == 0 ? (size_t)n * 2 * sizeof(float) : 0);
}

template <int TYPE>
struct Backward {
  NormGrads g;
  hipStream_t st;
  template <int G, int P>
  void run() const {
    norm_grads_kernel<TYPE, G, P><<<(unsigned)blocks_for(g.n, G, 4), 256, 0, st>>>(g);
  }
};

template <int TYPE>
void backward(const NormGrads& g, hipStream_t st) {
  if (with_shape(g.q, Backward<TYPE>{g, st})) return;
  norm_grads_rows_kernel<TYPE><<<(unsigned)g.n, LONG, 0, st>>>(g);
  norm_grads_columns_kernel<TYPE><<<dim3((g.q + 2047) / 2048, grads_groups(g.n, g.q)), 256, 0, st>>>(g);
}

bool known16(int type) { return type == OZGEMM_F32 || type == OZGEMM_BF16 || type == OZGEMM_F16; }

// Whether two arrays of rows may not both be used: one is written, they share
// memory and are not the same array.
bool clash(const void* a, size_t abytes, long lda, const void* b, size_t bbytes, long ldb) {
  return overlap(a, abytes, b, bbytes) && !(a == b && lda == ldb);
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

int ozgemm_rms_norm(int type, int ytype, int wtype, int n, int q, const void* X, int ldx, const void* R, int ldr,
                    const void* w, double eps, void* H, int ldh, void* Y, int ldy, float* S, long long srow,
                    long long sblock, void* hip_stream) {
  if (!known16(type)) return -1;
  const bool eight = ytype == OZGEMM_E4M3 || ytype == OZGEMM_E5M2;
  if (ytype != type && !eight) return -2;
  if (wtype != type && wtype != OZGEMM_F32) return -3;
  if (n < 0) return -4;
  if (q < 0) return -5;
  const bool any = n > 0 && q > 0;
  if (X == nullptr && any) return -6;
  if (ldx < std::max(1, q)) return -7;
  if (R != nullptr && ldr < std::max(1, q)) return -9;
  if (w == nullptr && any) return -10;
  if (!(eps >= 0.0)) return -11;
  if (R != nullptr && H == nullptr && any) return -12;
  if (R != nullptr && ldh < std::max(1, q)) return -13;
  if (Y == nullptr && any) return -14;
  if (ldy < std::max(1, q)) return -15;
  if (eight && S == nullptr && any) return -16;
  if (eight && srow < 0) return -17;
  if (eight && sblock < 0) return -18;
  if (n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return OZGEMM_RANGE;
  if (!any) return OZGEMM_OK;
  if (eight && !places_differ(n, (q - 1) / BLOCK8 + 1, srow, sblock)) return -17;
  const size_t size = elem_bytes(type);
  const size_t xb = extent(q, n, ldx, 0, 1, size), rb = R ? extent(q, n, ldr, 0, 1, size) : 0;
  const size_t wb = (size_t)q * elem_bytes(wtype), hb = R ? extent(q, n, ldh, 0, 1, size) : 0;
  const size_t yb = extent(q, n, ldy, 0, 1, eight ? 1 : size);
  const size_t sb =
      eight ? ((size_t)(n - 1) * srow + (size_t)((q - 1) / BLOCK8) * sblock + 1) * sizeof(float) : 0;
  if (clash(H, hb, ldh, X, xb, ldx) || clash(H, hb, ldh, R, rb, ldr) || overlap(H, hb, w, wb)) return -12;
  if ((eight ? overlap(Y, yb, X, xb) || overlap(Y, yb, R, rb)
             : clash(Y, yb, ldy, X, xb, ldx) || clash(Y, yb, ldy, R, rb, ldr)) ||
      overlap(Y, yb, H, hb) || overlap(Y, yb, w, wb))
    return -14;
  if (overlap(S, sb, X, xb) || overlap(S, sb, R, rb) || overlap(S, sb, H, hb) || overlap(S, sb, w, wb) ||
      overlap(S, sb, Y, yb))
    return -16;
  const Norm g{X, R, w, H, Y, S, ldx, ldr, ldh, ldy, (long)srow, (long)sblock, n, q, wtype == OZGEMM_F32, eps};
  hipStream_t st = (hipStream_t)hip_stream;
  if (type == OZGEMM_F32)
    forward_type<OZGEMM_F32>(ytype, g, st);
  else if (type == OZGEMM_BF16)
    forward_type<OZGEMM_BF16>(ytype, g, st);
  else
    forward_type<OZGEMM_F16>(ytype, g, st);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}

size_t ozgemm_rms_norm_grads_workspace_bytes(int n, int q, int dw) {
  if (n <= 0 || q <= 0 || n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return 0;
  return grads_workspace(n, q, dw != 0);
}

int ozgemm_rms_norm_grads(int type, int wtype, int n, int q, const void* dY, int lddy, const void* H, int ldh,
                          const void* w, const void* dH, int lddh, double eps, void* dX, int lddx, void* dw,
                          void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!known16(type)) return -1;
  if (wtype != type && wtype != OZGEMM_F32) return -2;
  if (n < 0) return -3;
  if (q < 0) return -4;
  const bool any = n > 0 && q > 0;
  if (dY == nullptr && any) return -5;
  if (lddy < std::max(1, q)) return -6;
  if (H == nullptr && any) return -7;
  if (ldh < std::max(1, q)) return -8;
  if (w == nullptr && any) return -9;
  if (dH != nullptr && lddh < std::max(1, q)) return -11;
  if (!(eps >= 0.0)) return -12;
  if (dX == nullptr && any) return -13;
  if (lddx < std::max(1, q)) return -14;
  if (n > OZGEMM_MAX_ROWS || q > OZGEMM_MAX_ROWS) return OZGEMM_RANGE;
  if (q == 0) return OZGEMM_OK;
  const size_t size = elem_bytes(type), wb = (size_t)q * elem_bytes(wtype), dwb = dw ? wb : 0;
  const size_t yb = extent(q, n, lddy, 0, 1, size), hb = extent(q, n, ldh, 0, 1, size);
  const size_t dhb = dH ? extent(q, n, lddh, 0, 1, size) : 0, xb = extent(q, n, lddx, 0, 1, size);
  if (clash(dX, xb, lddx, dY, yb, lddy) || clash(dX, xb, lddx, H, hb, ldh) || clash(dX, xb, lddx, dH, dhb, lddh) ||
      overlap(dX, xb, w, wb))
    return -13;
  if (overlap(dw, dwb, dY, yb) || overlap(dw, dwb, H, hb) || overlap(dw, dwb, dH, dhb) || overlap(dw, dwb, w, wb) ||
      overlap(dw, dwb, dX, xb))
    return -15;
  hipStream_t st = (hipStream_t)hip_stream;
  const int groups = any ? grads_groups(n, q) : 0;
  if (any) {
    const size_t need = grads_workspace(n, q, dw != nullptr);
    if (need > 0 && (workspace == nullptr || ((uintptr_t)workspace & 255))) return -16;
    if (workspace_bytes < need) return OZGEMM_WORKSPACE_TOO_SMALL;
    char* ws = (char*)workspace;
    const NormGrads g{dY,   H,    w,   dH,   dX, dw != nullptr ? (float*)ws : nullptr,
                      (float*)(ws + (dw != nullptr ? grads_partial_bytes(n, q) : 0)),
                      lddy, ldh,  lddh, lddx, n,  q, wtype == OZGEMM_F32, eps};
    if (type == OZGEMM_F32)
      backward<OZGEMM_F32>(g, st);
    else if (type == OZGEMM_BF16)
      backward<OZGEMM_BF16>(g, st);
    else
      backward<OZGEMM_F16>(g, st);
  }
  if (dw != nullptr)
    join_weights_kernel<<<(unsigned)((q + 31) / 32), 1024, 0, st>>>((const float*)workspace, groups, q, dw, wtype);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}

}  // extern "C"
