// Reads "a b c t" lines; prints the bounds of a step's states, their grids'
// exponents and the factors of its products.  With an argument: "norm eps"
// lines, and the first bound of each.
#include <cstdio>

#include "../fp64_gemm_emulation_ozii_amd/csrc/scales.h"

int main(int argc, char**) {
  double a, b, c, t;
  if (argc > 1) {
    while (std::scanf("%lf %lf", &a, &b) == 2) std::printf("%.17g\n", oz::first_bound(a, b));
    return 0;
  }
  while (std::scanf("%lf %lf %lf %lf", &a, &b, &c, &t) == 4) {
    const oz::Bends s = oz::bends_of(a, b, c);
    const oz::Bounds r = oz::advance(s, t);
    const oz::Factors f = oz::factors_of(s, r);
    std::printf("%.17g %.17g %.17g %.17g %d %d %d %d %.17g %.17g %.17g %.17g %.17g %d\n", r.X, r.P, r.Q, r.next,
                oz::grid_exponent(r.X), oz::grid_exponent(r.P), oz::grid_exponent(r.Q), f.next, f.f[0], f.f[1], f.g[1],
                f.f[2], f.g[2], (int)oz::in_range(r));
  }
}
