// The grids of a Newton-Schulz iteration's states (host and device code; a CPU
// test driver builds it too).
//
// A state lies in half slices as x 2^E, with E from a bound on |x|: the
// singular values of X_0 are at most t_0 = |G|_F / (|G|_F + eps), which may be
// anything down to 0, and those of the iterate at most
//   t' = max over [0, t] of |p|,  p(x) = a x + b x^3 + c x^5,
// those of P at most t^2, of Q = b P + c P^2 at most max over [0, t^2] of
// |b y + c y^2|.  Every matrix of a batch has grids of its own, since |G|_F is
// its own (with t_0 = 1 for all of them, entries of X_0 below 2^-26 of eps
// fell out of half's normal range).  Where p bends does not depend on t: `Bends`
// has it, one for each step, and a step of `advance` is a few multiplications.
#pragma once

#include <math.h>

#ifndef __HIPCC__
#ifndef __host__
#define __host__
#endif
#ifndef __device__
#define __device__
#endif
#endif

namespace oz {

struct Bends {
  double a, b, c;
  double y[2], top[2];  // x^2 of p's stationary points (0: none), and |p| there
  double yq, topq;      // the same of b y + c y^2
};

__host__ __device__ inline double odd_quintic(double a, double b, double c, double x) {
  return fabs(x * (a + x * x * (b + x * x * c)));
}

__host__ __device__ inline Bends bends_of(double a, double b, double c) {
  Bends s{a, b, c, {0, 0}, {0, 0}, 0, 0};
  if (c != 0) {  // a + 3 b y + 5 c y^2 = 0, without the difference that loses the small root where c is
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      const double h = -0.5 * (3 * b + copysign(sqrt(d), b));
      s.y[0] = h / (5 * c);
      if (h != 0) s.y[1] = a / h;
    }
    s.yq = -b / (2 * c);
    s.topq = fabs(b * b / (4 * c));
  } else if (b != 0) {
    s.y[0] = -a / (3 * b);
  }
  for (int i = 0; i < 2; ++i) {
    if (!(s.y[i] > 0)) s.y[i] = 0;
    s.top[i] = odd_quintic(a, b, c, sqrt(s.y[i]));
  }
  if (!(s.yq > 0)) s.yq = 0;
  return s;
}

// Bounds of a step's states: X, P, Q and the next X.
struct Bounds {
  double X, P, Q, next;
};

// The bounds hold for the exact iteration; rounding is left a 1024th of the
// next one.  They carry no further margin, because the polynomials of a schedule
// grow steeply past the interval they are made for and every bit given away
// here is lost to the low slices.
__host__ __device__ inline Bounds advance(const Bends& s, double t) {
  const double u = t * t;
  Bounds r{t, u, fabs(u * (s.b + s.c * u)), odd_quintic(s.a, s.b, s.c, t)};
  for (int i = 0; i < 2; ++i)
    if (s.y[i] > 0 && s.y[i] < u) r.next = fmax(r.next, s.top[i]);
  if (s.yq > 0 && s.yq < u) r.Q = fmax(r.Q, s.topq);
  r.next *= 1 + 1.0 / 1024;
  return r;
}

constexpr double BOUND_MAX = 1e18;  // the host refuses schedules that may pass it

__host__ __device__ inline bool in_range(const Bounds& r) {
  return r.X < BOUND_MAX && r.P < BOUND_MAX && r.Q < BOUND_MAX && r.next < BOUND_MAX;
}

// E with bound 2^E in [2^13, 2^14): an entry may pass the bound four times over
// before it leaves half's range (65504).  Below 2^-1000 nothing is left that a
// result could hold.
__host__ __device__ inline int grid_exponent(double bound) {
  int e = 0;
  frexp(fmax(bound, 0x1p-1000), &e);
  return 14 - e;
}

// t_0 of a matrix; 1 where the norm says nothing (zero, Inf or NaN).
__host__ __device__ inline double first_bound(double norm, double eps) {
  return norm > 0 && norm < HUGE_VAL ? fmax(norm / (norm + eps), 0x1p-400) : 1.0;
}

// A step's products on the grids: P = f[0] X X^T, Q = f[1] P P + g[1] P,
// X' = f[2] Q X + g[2] X, each of them within single precision's normal range or
// (f) too small beside the other term to matter.  `next`: X's exponent after it.
struct Factors {
  float f[3], g[3];
  int next;
};

__host__ __device__ inline Factors factors_of(const Bends& s, const Bounds& r) {
  const int x = grid_exponent(r.X), p = grid_exponent(r.P), q = grid_exponent(r.Q), n = grid_exponent(r.next);
  return Factors{{(float)ldexp(1.0, p - 2 * x), (float)ldexp(s.c, q - 2 * p), (float)ldexp(1.0, n - q - x)},
                 {0.f, (float)ldexp(s.b, q - p), (float)ldexp(s.a, n - x)},
                 n};
}

}  // namespace oz
