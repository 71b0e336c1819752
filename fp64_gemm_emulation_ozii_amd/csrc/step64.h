// The FP64 products of a Newton-Schulz step on the FP64 matrix cores, for
// matrices too small for Scheme II's passes to pay (ortho.hip has the rule):
//   v = alpha sum over k of A(i, k) B(j, k) + beta S[j][i]  ->  N[j][i]
// v_mfma_f64_16x16x4_f64 takes 64 cycles on a SIMD (32 operations per cycle), so
// one 16 x 16 tile's operands, 1 KB, feed it for as long as the LDS needs for
// several of them: the kernel is bound by the matrix cores, and at small sizes
// by the latency of its few K slabs.  Five steps on one matrix of 512 x 512 take
// 248 us (13 us a product), on 520 x 3688 0.95 ms (25 TFLOPS).
#pragma once

#include <hip/hip_runtime.h>

#include "tile16.h"

namespace oz {

struct Step64 {
  const double* A;  // entry (i, k) at i a_i + k a_k, one of them 1
  const double* B;
  long a_i, a_k, b_j, b_k, a_batch, b_batch;
  int m, n, k, batch;
  double alpha, beta;
  const double* S;  // [j][i], rows s_ld apart; nullptr: none
  long s_ld, s_batch;
  double* N;        // [j][i], rows n_ld apart
  long n_ld, n_batch;
};

template <int BT, int KS, bool SYM>
__global__ __launch_bounds__(256) void step64_kernel(Step64 p) {
  constexpr int PITCH = BT + 2, F = BT / 32;  // a wavefront has F x F tiles of 16 x 16
  constexpr int PER = BT * KS / 256;          // entries of a slab per thread
  typedef double v4d __attribute__((ext_vector_type(4)));
  __shared__ double sa[2][KS][PITCH], sb[2][KS][PITCH];
  const int tm = (p.m + BT - 1) / BT, tn = (p.n + BT - 1) / BT;
  const int per = SYM ? tm * (tm + 1) / 2 : tm * tn;
  const int w = xcd_order(blockIdx.x, per * p.batch);
  const long b = w / per;
  int mi, nj;
  if (SYM)
    triangle_order<4>(w % per, tm, mi, nj);
  else
    panel_order<4>(w % per, tm, tn, mi, nj);
  const int m0 = mi * BT, n0 = nj * BT;
  const double* A = p.A + b * p.a_batch;
  const double* B = p.B + b * p.b_batch;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * (BT / 2), wn = (wave >> 1) * (BT / 2);
  // Entry e of this thread in a slab: neighbouring threads along the
  // contiguous index.  A row past the end reads row 0 and keeps zero.
  const bool ak = p.a_k == 1, bk = p.b_k == 1;
  const double* pa[PER];
  const double* pb[PER];
  int ka[PER], kb[PER];
  double* da[PER];
  double* db[PER];
  bool ia[PER], ib[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int at = e * 256 + threadIdx.x;
    int row = ak ? at / KS : at % BT;
    ka[e] = ak ? at % KS : at / BT;
    ia[e] = m0 + row < p.m;
    da[e] = &sa[0][ka[e]][row];
    pa[e] = A + (ia[e] ? (m0 + row) * p.a_i : 0) + ka[e] * p.a_k;
    row = bk ? at / KS : at % BT;
    kb[e] = bk ? at % KS : at / BT;
    ib[e] = n0 + row < p.n;
    db[e] = &sb[0][kb[e]][row];
    pb[e] = B + (ib[e] ? (n0 + row) * p.b_j : 0) + kb[e] * p.b_k;
  }
  double ra[PER], rb[PER];
  auto load = [&](int k0) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      ra[e] = k0 + ka[e] < p.k ? *pa[e] : 0.0;
      rb[e] = k0 + kb[e] < p.k ? *pb[e] : 0.0;
      pa[e] += KS * p.a_k;
      pb[e] += KS * p.b_k;
    }
  };
  auto keep = [&](int buf) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      da[e][buf * KS * PITCH] = ia[e] ? ra[e] : 0.0;
      db[e][buf * KS * PITCH] = ib[e] ? rb[e] : 0.0;
    }
  };
  // rows of the MFMA's result are j, its columns i: 16 lanes hold i next to each other
  v4d acc[F][F] = {};
  load(0);
  keep(0);
  __syncthreads();
  for (int k0 = 0, buf = 0; k0 < p.k; k0 += KS, buf ^= 1) {
    const bool more = k0 + KS < p.k;
    if (more) load(k0 + KS);
#pragma unroll
    for (int kk = 0; kk < KS; kk += 4) {
      double fa[F], fb[F];
#pragma unroll
      for (int f = 0; f < F; ++f) {
        fa[f] = sa[buf][kk + (lane >> 4)][wm + f * 16 + (lane & 15)];
        fb[f] = sb[buf][kk + (lane >> 4)][wn + f * 16 + (lane & 15)];
      }
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int i = 0; i < F; ++i) acc[j][i] = __builtin_amdgcn_mfma_f64_16x16x4f64(fb[j], fa[i], acc[j][i], 0, 0, 0);
    }
    if (more) keep(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < F; ++j)
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int col = n0 + wn + j * 16 + 4 * r + (lane >> 4), row = m0 + wm + i * 16 + (lane & 15);
        if (col >= p.n || row >= p.m) continue;
        double v = p.alpha * acc[j][i][r];
        if (p.S != nullptr) v = __builtin_fma(p.beta, p.S[b * p.s_batch + col * p.s_ld + row], v);
        p.N[b * p.n_batch + col * p.n_ld + row] = v;
        if (SYM && m0 != n0) p.N[b * p.n_batch + row * p.n_ld + col] = v;
      }
}

template <int BT, int KS>
hipError_t launch_step64_t(const Step64& p, bool sym, long blocks, hipStream_t st) {
  if (sym)
    hipLaunchKernelGGL((step64_kernel<BT, KS, true>), dim3((unsigned)blocks), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((step64_kernel<BT, KS, false>), dim3((unsigned)blocks), dim3(256), 0, st, p);
  return hipGetLastError();
}

// 32 x 32 tiles (larger ones leave the compute units idle at the sizes that
// come here: 1024^2 0.91 ms, with 64 x 64 tiles 1.18).  Up to two blocks per
// unit wait for their loads, and K slabs of 64 keep four times as many in
// flight as slabs of 16 (512^2: 0.29 against 0.38 ms); more blocks hide them
// for each other, and small slabs let more run (4 x 512 x 1024: 0.73 against 0.87 ms).
inline hipError_t launch_step64(const Step64& p, bool sym, int units, hipStream_t st) {
  const long tm = (p.m + 31) / 32, tn = (p.n + 31) / 32;
  const long blocks = (sym ? tm * (tm + 1) / 2 : tm * tn) * p.batch;
  return blocks <= 2L * units ? launch_step64_t<32, 64>(p, sym, blocks, st) : launch_step64_t<32, 16>(p, sym, blocks, st);
}

}  // namespace oz
