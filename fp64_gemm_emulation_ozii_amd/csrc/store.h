// Where the accumulators of a tile of products go (gemm16.hip, gemm8.h).
#pragma once

#include "tile16.h"

namespace oz {

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
// would write 8-byte pieces of 16 different columns.)  The caller has seen to
// it that nobody uses the pieces.
template <class Tile>
struct Store {
  static constexpr int WTM = Tile::FM * 16, PITCH = WTM + 4, RUNS = WTM / 8, CH = 16 * RUNS / 64;
  static constexpr int BYTES = Tile::NW * 16 * PITCH * 4;
  static_assert(16 * RUNS % 64 == 0, "whole wavefronts of runs");

  // 16-byte stores of every wavefront, in STORES, where every lane stores
  // every run of a tile; 0 where some do not.
  static __device__ __forceinline__ int stores(const Target& t, int bm, int bn) {
    const bool all = t.m0 + bm <= t.m && t.n0 + bn <= t.n_end;
    return !all ? 0 : t.ctype == OZGEMM_F32 ? 2 : 1;
  }
  static constexpr int STORES = Tile::FN * CH;

  static __device__ __forceinline__ void run(const v4f (&acc)[Tile::FM][Tile::FN], char* smem, const Target& t) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* stage = reinterpret_cast<float*>(smem) + wave * 16 * PITCH;
    const int mw = t.m0 + Tile::wave_m(wave) * WTM, nw = t.n0 + Tile::wave_n(wave) * (Tile::FN * 16);
    const int size = t.ctype == OZGEMM_F32 ? 4 : 2;
    // a lane's runs all begin at the same row
    static_assert(64 % RUNS == 0, "a lane keeps its rows");
    const int row = mw + lane % RUNS * 8;
    int ea[8] = {};
    if (t.ea != nullptr) {
#pragma unroll
      for (int k = 0; k < 8; ++k) ea[k] = t.ea[min(row + k, t.m - 1)];
    }
#pragma unroll
    for (int j = 0; j < Tile::FN; ++j) {
      int eb[CH] = {};
      if (t.ea != nullptr) {
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) eb[ch] = t.eb[min(nw + j * 16 + (ch * 64 + lane) / RUNS, t.n_end - 1)];
      }
#pragma unroll
      for (int i = 0; i < Tile::FM; ++i)
        *reinterpret_cast<v4f*>(stage + (lane & 15) * PITCH + i * 16 + 4 * (lane >> 4)) = acc[i][j];
      __builtin_amdgcn_s_waitcnt(0xc07f);  // the wave's own writes; no other wave uses this piece
      asm volatile("" ::: "memory");
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const int at = ch * 64 + lane, c = at / RUNS, r = at % RUNS * 8;
        const int col = nw + j * 16 + c;
        if (col >= t.n_end || row >= t.m) continue;
        float v[8];
        *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r);
        *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(stage + c * PITCH + r + 4);
        if (t.ea != nullptr) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = unscale(v[k], ea[k], eb[ch]);
        }
        char* out = (char*)t.C + ((long)col * t.ldc + row) * size;
        const bool all = row + 8 <= t.m;
        if (t.ctype == OZGEMM_F32) {
          if (all) {
            *reinterpret_cast<v4f_any*>(out) = v4f{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<v4f_any*>(out + 16) = v4f{v[4], v[5], v[6], v[7]};
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (row + k < t.m) reinterpret_cast<float*>(out)[k] = v[k];
          }
        } else {
          v8s h;
#pragma unroll
          for (int k = 0; k < 8; ++k) h[k] = (short)round16(v[k], t.ctype);
          if (all) {
            *reinterpret_cast<v8s_any*>(out) = h;
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
};

}  // namespace oz
