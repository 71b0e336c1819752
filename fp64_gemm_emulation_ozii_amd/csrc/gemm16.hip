// Products over ragged groups in 16-bit slices (tile16.h).
//
//   grouped:  C(:, j) = op(A_e) B(:, j)          for j in J_e
//   outer:    C_e = sum over j in J_e of A(:, j) B(:, j)^T
//
// J_e are the groups of groups.h, known on the device only: a launch has a
// block for every tile the groups could need, and each block looks its tile
// up in the offsets (one wavefront-wide scan per 64 groups).
#include "groups.h"
#include "products.h"
#include "tile16.h"

namespace oz {

namespace {

// x rounded to a 16-bit type, to nearest-even.
__device__ __forceinline__ uint16_t round16(float x, int ctype) {
  return ctype == OZGEMM_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
                              : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// acc 2^(ea + eb - 30): the slices of a row lie on a grid whose largest entry is
// below 2^15 (slices.hip).  One rounding (v_ldexp_f32); a row that holds Inf or NaN gives NaN.
__device__ __forceinline__ float unscale(float x, int ea, int eb) {
  if (ea == OZGEMM_EXP_NONFINITE || eb == OZGEMM_EXP_NONFINITE) return __builtin_nanf("");
  return __builtin_ldexpf(x, ea + eb - 30);
}

// Where a tile's accumulators go: rows [m0, m) x columns [n0, n_end) of C,
// row exponents ea and column exponents eb (nullptr: none).
struct Target {
  void* C;
  int ctype;
  long ldc;
  int m0, m, n0, n_end;
  const int32_t* ea;
  const int32_t* eb;
};

// Each wavefront passes its accumulators 16 columns at a time through a piece
// of LDS of its own and writes runs of 8 rows: 16 or 32 bytes per lane, a
// column's runs next to each other.  (From the accumulators themselves a lane
// would write 8-byte pieces of 16 different columns.)
template <class Tile>
__device__ __forceinline__ void store_tile(const v4f (&acc)[Tile::FM][Tile::FN], char* smem, const Target& t) {
  constexpr int WTM = Tile::FM * 16, PITCH = WTM + 4, RUNS = WTM / 8;
  static_assert(Tile::NW * 16 * PITCH * 4 <= Tile::SMEM, "staging fits the operand buffers");
  slice_barrier<0>();  // every wave has read its last operands
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* stage = reinterpret_cast<float*>(smem) + wave * 16 * PITCH;
  const int mw = t.m0 + wave / Tile::WAVES_N * WTM, nw = t.n0 + wave % Tile::WAVES_N * (Tile::FN * 16);
  const int size = t.ctype == OZGEMM_F32 ? 4 : 2;
  const bool wide = (t.ldc & 7) == 0 && ((uintptr_t)t.C & 15) == 0;
#pragma unroll
  for (int j = 0; j < Tile::FN; ++j) {
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
      *reinterpret_cast<v4f*>(stage + (lane & 15) * PITCH + i * 16 + 4 * (lane >> 4)) = acc[i][j];
    __builtin_amdgcn_s_waitcnt(0xc07f);  // the wave's own writes; no other wave uses this piece
    asm volatile("" ::: "memory");
#pragma unroll 1
    for (int at = lane; at < 16 * RUNS; at += 64) {
      const int c = at / RUNS, r = at % RUNS * 8;
      const int col = nw + j * 16 + c, row = mw + r;
      if (col >= t.n_end || row >= t.m) continue;
      float v[8];
      *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r);
      *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r + 4);
      if (t.ea != nullptr) {
        const int eb = t.eb[col];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = unscale(v[k], t.ea[min(row + k, t.m - 1)], eb);
      }
      char* out = (char*)t.C + ((long)col * t.ldc + row) * size;
      const bool whole = wide && row + 8 <= t.m;
      if (t.ctype == OZGEMM_F32) {
        if (whole) {
          *reinterpret_cast<v4f*>(out) = v4f{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<v4f*>(out + 16) = v4f{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (row + k < t.m) reinterpret_cast<float*>(out)[k] = v[k];
        }
      } else {
        v8s h;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = (short)round16(v[k], t.ctype);
        if (whole) {
          *reinterpret_cast<v8s*>(out) = h;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (row + k < t.m) reinterpret_cast<short*>(out)[k] = h[k];
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
  }
}

template <class T, int BM, int BN, int WM, int WN, bool AKS, bool PAIR>
__global__ __launch_bounds__(WM* WN * 64) void grouped_n_kernel(Grouped16 g) {
  using Tile = Tile16<T, BM, BN, WM, WN, AKS, false, 2, PAIR>;
  __shared__ __attribute__((aligned(1024))) char smem[Tile::SMEM];
  const int tiles_m = (g.m + BM - 1) / BM;
  const int tiles_n = count_group_tiles(g.offsets, g.groups, g.n, BN);
  const long total = (long)tiles_m * tiles_n;
  if (blockIdx.x >= total) return;
  int nj, mi;
  panel_order<4>(xcd_order(blockIdx.x, (int)total), tiles_n, tiles_m, nj, mi);
  const GroupTile gt = find_group_tile(g.offsets, g.groups, g.n, BN, nj);
  if (gt.group < 0) return;
  const int m0 = mi * BM, n0 = gt.begin;
  Source16 A, B;
  A.ld = (int)g.A.ld;
  A.plane = g.A.plane;
  A.base = g.A.p + gt.group * g.A.batch + (AKS ? (long)m0 : (long)m0 * g.A.ld);
  A.rows = g.m - m0;
  A.last = (int)g.A.last - (AKS ? m0 : 0);
  B.ld = (int)g.B.ld;
  B.plane = g.B.plane;
  B.base = g.B.p + (long)n0 * g.B.ld;
  B.rows = g.n - n0;
  B.last = (int)g.B.last;
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, A, B, g.q);
  store_tile<Tile>(acc, smem,
                   Target{g.C, g.ctype, g.ldc, m0, g.m, n0, gt.end,
                          g.A.ex ? g.A.ex + gt.group * g.A.ex_batch : nullptr, g.B.ex});
}

template <class T, int BM, int BN, int WM, int WN, bool KS, bool PAIR>
__global__ __launch_bounds__(WM* WN * 64) void grouped_k_kernel(Grouped16 g) {
  using Tile = Tile16<T, BM, BN, WM, WN, KS, KS, 2, PAIR>;
  __shared__ __attribute__((aligned(1024))) char smem[Tile::SMEM];
  const int tiles_m = (g.m + BM - 1) / BM, tiles_q = (g.q + BN - 1) / BN;
  const int per = tiles_m * tiles_q;
  const int w = xcd_order(blockIdx.x, per * g.groups);
  int mi, qj;
  panel_order<4>(w % per, tiles_m, tiles_q, mi, qj);
  const int e = w / per;
  const GroupTile gt = group_at(g.offsets, g.groups, g.n, BK16, e);
  const int len = gt.end - gt.begin;
  const int m0 = mi * BM, q0 = qj * BN;
  Source16 A, B;
  A.ld = (int)g.A.ld;
  A.plane = g.A.plane;
  B.ld = (int)g.B.ld;
  B.plane = g.B.plane;
  A.rows = g.m - m0;
  B.rows = g.q - q0;
  int inner = len;
  if (KS) {
    A.base = g.A.p + gt.begin * g.A.ld + m0;
    A.last = (int)g.A.last - m0;
    B.base = g.B.p + gt.begin * g.B.ld + q0;
    B.last = (int)g.B.last - q0;
  } else {  // padded planes: the group's rows begin at 64 x its tiles before
    const int k0 = gt.first * BK16;
    inner = (len + BK16 - 1) / BK16 * BK16;
    A.base = g.A.p + (long)m0 * g.A.ld + k0;
    A.last = (int)g.A.last - k0;
    B.base = g.B.p + (long)q0 * g.B.ld + k0;
    B.last = (int)g.B.last - k0;
  }
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, A, B, inner);
  char* C = (char*)g.C + (size_t)e * g.cbatch * (g.ctype == OZGEMM_F32 ? 4 : 2);
  store_tile<Tile>(acc, smem,
                   Target{C, g.ctype, g.ldc, m0, g.m, q0, g.q, g.A.ex ? g.A.ex + e * g.A.ex_batch : nullptr,
                          g.B.ex ? g.B.ex + e * g.B.ex_batch : nullptr});
}

template <class T, int BT, bool AKS, bool PAIR>
hipError_t grouped_n(const Grouped16& g, hipStream_t st) {
  const long blocks = group_tiles_max(g.n, g.groups, BT) * ((g.m + BT - 1) / BT);
  hipLaunchKernelGGL((grouped_n_kernel<T, BT, BT, 2, 4, AKS, PAIR>), dim3((unsigned)blocks), dim3(512), 0, st, g);
  return hipGetLastError();
}

template <class T, int BT, bool KS, bool PAIR>
hipError_t grouped_k(const Grouped16& g, hipStream_t st) {
  const long blocks = (long)((g.m + BT - 1) / BT) * ((g.q + BT - 1) / BT) * g.groups;
  hipLaunchKernelGGL((grouped_k_kernel<T, BT, BT, 2, 4, KS, PAIR>), dim3((unsigned)blocks), dim3(512), 0, st, g);
  return hipGetLastError();
}

}  // namespace

// counted with the smallest tiles any variant uses
bool grouped_n_fits(const Grouped16& g) {
  return group_tiles_max(g.n, g.groups, 64) * ((g.m + 63) / 64) <= 0x7fffffffL;
}

bool grouped_k_fits(const Grouped16& g) {
  return (long)((g.m + 63) / 64) * ((g.q + 63) / 64) <= 0x7fffffffL / g.groups;
}

hipError_t launch_grouped_n(const Grouped16& g, hipStream_t st) {
  if (g.B.ks || (g.f32 && g.A.ks)) return hipErrorInvalidValue;
  if (g.f32) return grouped_n<Half, 128, false, true>(g, st);
  if (g.bf16) return g.A.ks ? grouped_n<Bfloat, 256, true, false>(g, st) : grouped_n<Bfloat, 256, false, false>(g, st);
  return g.A.ks ? grouped_n<Half, 256, true, false>(g, st) : grouped_n<Half, 256, false, false>(g, st);
}

hipError_t launch_grouped_k(const Grouped16& g, hipStream_t st) {
  if (g.A.ks != g.B.ks || (g.f32 && g.A.ks)) return hipErrorInvalidValue;
  if (g.f32) return grouped_k<Half, 128, false, true>(g, st);
  if (g.bf16) return g.A.ks ? grouped_k<Bfloat, 256, true, false>(g, st) : grouped_k<Bfloat, 256, false, false>(g, st);
  return g.A.ks ? grouped_k<Half, 256, true, false>(g, st) : grouped_k<Half, 256, false, false>(g, st);
}

}  // namespace oz
