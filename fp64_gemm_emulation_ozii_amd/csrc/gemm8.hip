// Products of 8-bit operands in scaled blocks (gemm8.h) on gfx950 matrix cores.
//
// Two ways to sum a block's 128 products:
//   narrow  one v_mfma_f32_16x16x128_f8f6f4, for results of 16 bits.  Within the
//           products that one lane holds the matrix core keeps what lies above
//           2^-13 of the largest: blocks of gaussian entries come out with an
//           error of 1.5e-5 of their sum's norm, a fifteenth of float16's
//           rounding and a hundredth of bfloat16's.
//   wide    four v_mfma_f32_16x16x32_f16 of the same entries as half precision
//           (both 8-bit types are exact there), for float32 results: the sums are
//           float32 throughout, at half the rate.
// A block's sum is then multiplied by its scales and added to the accumulators
// in float32.
#include <algorithm>

#include "block8.h"
#include "gemm8.h"
#include "products.h"
#include "store.h"
#include "tile16.h"

namespace oz {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Two of a word's four 8-bit values as halves (exact).
template <int TYPE, bool HIGH>
__device__ __forceinline__ uint32_t halves(uint32_t w) {
  if constexpr (TYPE == OZGEMM_E4M3) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HIGH));
  } else {  // e5m2 is the upper byte of a half
    return HIGH ? __builtin_amdgcn_perm(0u, w, 0x030c020cu) : __builtin_amdgcn_perm(0u, w, 0x010c000cu);
  }
}

template <int TYPE>
__device__ __forceinline__ v8h halves8(uint32_t lo, uint32_t hi) {
  const v4u8 w = {halves<TYPE, false>(lo), halves<TYPE, true>(lo), halves<TYPE, false>(hi), halves<TYPE, true>(hi)};
  return __builtin_bit_cast(v8h, w);
}

// 16 rows x 128 entries of an operand: lane l holds 32 of row l mod 16, the
// same ones for both operands (which ones does not matter to their product).
template <int TYPE, bool WIDE>
struct Frag;
template <int TYPE>
struct Frag<TYPE, false> {
  v8i w;
  __device__ __forceinline__ void set(v4u8 a, v4u8 b) {
    w = v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  }
};
template <int TYPE>
struct Frag<TYPE, true> {
  v8h h[4];
  __device__ __forceinline__ void set(v4u8 a, v4u8 b) {
    h[0] = halves8<TYPE>(a[0], a[1]);
    h[1] = halves8<TYPE>(a[2], a[3]);
    h[2] = halves8<TYPE>(b[0], b[1]);
    h[3] = halves8<TYPE>(b[2], b[3]);
  }
};

// A block's sums of 16 x 16 results: lane l has rows 4 (l / 16) .. + 3 of column l mod 16.
template <int TA, int TB, bool WIDE>
__device__ __forceinline__ v4f block_product(const Frag<TA, WIDE>& a, const Frag<TB, WIDE>& b) {
  v4f d = {0.f, 0.f, 0.f, 0.f};
  if constexpr (WIDE) {
#pragma unroll
    for (int t = 0; t < 4; ++t) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[t], b.h[t], d, 0, 0, 0);
  } else {
    // scales of 1 (a byte of 127) within the instruction
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.w, b.w, d, TA == OZGEMM_E5M2, TB == OZGEMM_E5M2, 0, 127, 0,
                                                         127);
  }
  return d;
}

// The bytes of a 16-byte piece at or past `left` as zeros.
__device__ __forceinline__ v4u8 first_bytes(v4u8 v, int left) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int bits = min(max(left - 4 * k, 0), 4) * 8;
    v[k] = bits == 32 ? v[k] : v[k] & ((1u << bits) - 1u);
  }
  return v;
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------

// BM x BN results by WM x WN wavefronts.  Blocks of 128 entries go from HBM
// straight into LDS through two buffers, 16 bytes per lane, range-checked (rows
// past the end arrive as zeros, as do pieces past the inner dimension), with
// their rows' scales beside them.
template <int TA, int TB, bool WIDE, bool AROW, int BM, int BN, int WM, int WN>
struct Tile8 {
  static constexpr int NW = WM * WN, THREADS = NW * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int ROWS = BM + BN;
  static constexpr int SCALES = ROWS * 4, BUF = ROWS * 128 + SCALES;
  static constexpr int LOADS = ROWS * 128 / 1024 / NW, A_LOADS = BM * 128 / 1024 / NW;
  static constexpr int SLOADS = (ROWS + THREADS - 1) / THREADS;
  static_assert(LOADS * NW * 1024 == ROWS * 128 && A_LOADS * NW * 1024 == BM * 128, "whole wave loads");
  static_assert(ROWS % THREADS == 0 && BM % 64 == 0, "whole wave loads of scales");
  static constexpr int wave_m(int wave) { return wave % WM; }
  static constexpr int wave_n(int wave) { return wave / WM; }
  static __device__ __forceinline__ int swz(int row) { return ((row >> 1) ^ (row << 2)) & 7; }

  static __device__ __forceinline__ void run(v4f (&acc)[FM][FN], char* smem, const Scaled8& g, int m0, int n0, int k0,
                                             int k_end) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave_m(wave), wn = wave_n(wave);
    // this lane's pieces: row r of 8, piece c, in loads of even and odd number
    int offa[2], offb[2], kin[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = lane >> 3, c = (lane & 7) ^ swz(e * 8 + r);
      kin[e] = c * 16;
      offa[e] = r * (int)g.A.ld + kin[e];
      offb[e] = r * (int)g.B.ld + kin[e];
    }
    const int rows_a = min(g.m - m0, BM), rows_b = min(g.n - n0, BN);
    const uint8_t* pa = g.A.p + (long)m0 * g.A.ld + k0;
    const uint8_t* pb = g.B.p + (long)n0 * g.B.ld + k0;
    // bytes from there to the end of the last row's last 16-byte piece
    const int len = (g.q + 15) / 16 * 16 - k0;
    int reca = (rows_a - 1) * (int)g.A.ld + len, recb = (rows_b - 1) * (int)g.B.ld + len;
    const float* ps[SLOADS];
    long sstep[SLOADS];
#pragma unroll
    for (int u = 0; u < SLOADS; ++u) {
      const int r = (u * NW + wave) * 64 + lane;
      const bool a = (u * NW + wave) * 64 < BM;
      const int row = a ? min(m0 + r, g.m - 1) >> g.A.shift : min(n0 + r - BM, g.n - 1);
      const Operand8& o = a ? g.A : g.B;
      sstep[u] = o.sblock;
      ps[u] = o.s + row * o.srow + (k0 >> 7) * o.sblock;
    }
    int left = k_end - k0;  // from the block to load on
    const int total = (left + 127) >> 7;
    auto issue = [&](int buf) {
      char* d = smem + buf * BUF;
      const __amdgpu_buffer_rsrc_t ra =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pa), 0, left > 0 ? reca : 0, 0x00020000);
      const __amdgpu_buffer_rsrc_t rb =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pb), 0, left > 0 ? recb : 0, 0x00020000);
#pragma unroll
      for (int li = 0; li < LOADS; ++li) {
        const bool a = li < A_LOADS;
        const int blk = a ? wave * A_LOADS + li : wave * (LOADS - A_LOADS) + li - A_LOADS;
        const int e = blk & 1;
        const int off = kin[e] < left ? (a ? offa[e] : offb[e]) : (int)0x80000000;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            a ? ra : rb, (__attribute__((address_space(3))) void*)(d + (a ? 0 : BM * 128) + blk * 1024), 16,
            off + blk * 8 * (int)(a ? g.A.ld : g.B.ld), 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < SLOADS; ++u) {
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)ps[u],
            (__attribute__((address_space(3))) void*)(d + ROWS * 128 + (u * NW + wave) * 256), 4, 0, 0);
        if (left > 128) ps[u] += sstep[u];
      }
      left -= 128;
      pa += 128;
      pb += 128;
      reca -= 128;
      recb -= 128;
    };
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    if (total > 0) issue(0);
    const int tail = (k_end - k0) & 15;  // bytes of the last piece of a row that count
    for (int t = 0; t < total; ++t) {
      char* buf = smem + (t & 1) * BUF;
      slice_barrier<0>();  // block t has landed, and everybody has read block t - 1
      if (t + 1 < total) issue((t + 1) & 1);
      if (t + 1 == total && tail != 0) {
        const int c = ((k_end - k0) & 127) >> 4;
        for (int r = threadIdx.x; r < ROWS; r += THREADS) {
          v4u8* at = reinterpret_cast<v4u8*>(buf + r * 128 + (c ^ swz(r)) * 16);
          *at = first_bytes(*at, tail);
        }
        __syncthreads();
      }
      auto piece = [&](int row, int h) {
        return *reinterpret_cast<const v4u8*>(buf + row * 128 + ((h * 4 + (lane >> 4)) ^ swz(row)) * 16);
      };
      const float* sa = reinterpret_cast<const float*>(buf + ROWS * 128);
      const float* sb = sa + BM;
      Frag<TB, WIDE> b[FN];
      float xb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn * (BN / WN) + j * 16 + (lane & 15);
        b[j].set(piece(BM + row, 0), piece(BM + row, 1));
        xb[j] = sb[row];
      }
      if (!AROW) {
        const float s = sa[wm * (BM / WM)];
#pragma unroll
        for (int j = 0; j < FN; ++j) xb[j] *= s;
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm * (BM / WM) + i * 16;
        Frag<TA, WIDE> a;
        a.set(piece(row + (lane & 15), 0), piece(row + (lane & 15), 1));
        v4f s4 = {1.f, 1.f, 1.f, 1.f};
        if (AROW) s4 = *reinterpret_cast<const v4f*>(sa + row + 4 * (lane >> 4));
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v4f d = block_product<TA, TB, WIDE>(a, b[j]);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = __builtin_fmaf(d[r], AROW ? s4[r] * xb[j] : xb[j], acc[i][j][r]);
        }
      }
    }
  }
};

template <class Tile, int BM, int BN>
__global__ __launch_bounds__(Tile::THREADS) void scaled_tiles_kernel(Scaled8 g) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tiles_m = (g.m + BM - 1) / BM, tiles_n = (g.n + BN - 1) / BN, whole = tiles_m * tiles_n;
  const int part = blockIdx.x / whole;
  int nj, mi;
  panel_order<4>(xcd_order(blockIdx.x - part * whole, whole), tiles_n, tiles_m, nj, mi);
  const int blocks = (g.q + 127) >> 7, each = (blocks + g.parts - 1) / g.parts;
  const int k0 = min(part * each, blocks) * 128, k_end = min(g.q, k0 + each * 128);
  v4f acc[Tile::FM][Tile::FN];
  Tile::run(acc, smem, g, mi * BM, nj * BN, k0, k_end);
  slice_barrier<0>();
  const Target to = g.parts > 1 ? Target{g.partial + (long)part * g.n * g.m, OZGEMM_F32, g.m, mi * BM, g.m, nj * BN,
                                         g.n, nullptr, nullptr}
                                : Target{g.C, g.ctype, g.ldc, mi * BM, g.m, nj * BN, g.n, nullptr, nullptr};
  Store<Tile>::run(acc, smem, to);
}

// The sum of the parts, in their order: a block per column and 1024 rows.
__global__ __launch_bounds__(256) void join_parts_kernel(Scaled8 g) {
  const int row = blockIdx.y * 1024 + threadIdx.x * 4;
  const long col = blockIdx.x;
  if (row >= g.m) return;
  const v4f v = sum_parts(g.partial + col * g.m + row, (long)g.n * g.m, g.parts, g.m - row);
  const long to = col * g.ldc + row;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (row + k >= g.m) break;
    if (g.ctype == OZGEMM_F32)
      ((float*)g.C)[to + k] = v[k];
    else
      ((uint16_t*)g.C)[to + k] = round16(v[k], g.ctype);
  }
}

// ---------------------------------------------------------------------------
// Few columns
// ---------------------------------------------------------------------------

constexpr int FEW8_WAVES = 8;

// Bound by reading A once: a block takes 16 MR rows of it and all (up to 16
// FN) columns; its eight wavefronts share the inner dimension block by block,
// straight from HBM into MFMA operands, and their sums meet in LDS.  The
// products are wide: next to the loads they cost nothing.
template <int TA, int TB, bool AROW, int MR, int FN>
__global__ __launch_bounds__(FEW8_WAVES * 64) void scaled_few_kernel(Scaled8 g) {
  __shared__ v4f sums[FEW8_WAVES][MR][FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = blockIdx.x * 16 * MR, piece = lane >> 4;
  const uint8_t* pa[MR];
  const uint8_t* pb[FN];
  const float* sb[FN];
#pragma unroll
  for (int i = 0; i < MR; ++i) pa[i] = g.A.p + (long)min(m0 + i * 16 + (lane & 15), g.m - 1) * g.A.ld + piece * 16;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int col = min(j * 16 + (lane & 15), g.n - 1);
    pb[j] = g.B.p + (long)col * g.B.ld + piece * 16;
    sb[j] = g.B.s + col * g.B.srow;
  }
  v4f acc[MR][FN] = {};
  const int blocks = (g.q + 127) >> 7;
#pragma unroll 2
  for (int b = wave; b < blocks; b += FEW8_WAVES) {
    const int k = b * 128, left = g.q - k - piece * 16;  // of this lane's first piece
    v4u8 ra[MR][2], rb[FN][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool any = left > h * 64;
#pragma unroll
      for (int i = 0; i < MR; ++i)
        ra[i][h] = any ? *reinterpret_cast<const v4u8*>(pa[i] + k + h * 64) : v4u8{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < FN; ++j)
        rb[j][h] = any ? *reinterpret_cast<const v4u8*>(pb[j] + k + h * 64) : v4u8{0, 0, 0, 0};
    }
    float xb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) xb[j] = sb[j][b * g.B.sblock];
    v4f s4[MR];
#pragma unroll
    for (int i = 0; i < MR; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = min(m0 + i * 16 + (AROW ? 4 * (lane >> 4) + r : 0), g.m - 1) >> g.A.shift;
        s4[i][r] = AROW || r == 0 ? g.A.s[row * g.A.srow + b * g.A.sblock] : s4[i][0];
      }
    }
    if (left < 128 && (g.q & 15) != 0) {  // a piece that ends inside the last block
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < MR; ++i) ra[i][h] = first_bytes(ra[i][h], left - h * 64);
#pragma unroll
        for (int j = 0; j < FN; ++j) rb[j][h] = first_bytes(rb[j][h], left - h * 64);
      }
    }
    Frag<TB, true> fb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j].set(rb[j][0], rb[j][1]);
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      Frag<TA, true> fa;
      fa.set(ra[i][0], ra[i][1]);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const v4f d = block_product<TA, TB, true>(fa, fb[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s4[i][r] * xb[j], acc[i][j][r]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sums[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  for (int u = threadIdx.x; u < MR * FN * 64; u += FEW8_WAVES * 64) {
    const int l = u & 63, j = u / 64 % FN, i = u / 64 / FN;
    v4f v = sums[0][i][j][l];
#pragma unroll
    for (int w = 1; w < FEW8_WAVES; ++w) v += sums[w][i][j][l];
    const int col = j * 16 + (l & 15), row = m0 + i * 16 + 4 * (l >> 4);
    if (col >= g.n) continue;
    const long to = col * g.ldc + row;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (row + r >= g.m) break;
      if (g.ctype == OZGEMM_F32)
        ((float*)g.C)[to + r] = v[r];
      else
        ((uint16_t*)g.C)[to + r] = round16(v[r], g.ctype);
    }
  }
}

__global__ __launch_bounds__(256) void align_rows_kernel(const uint8_t* src, long ld, int q, uint8_t* dst, long dld) {
  const int c = (blockIdx.y * 256 + threadIdx.x) * 16;
  if (c >= q) return;
  const uint8_t* p = src + blockIdx.x * ld + c;
  v4u8 v = {0, 0, 0, 0};
  if (c + 16 <= q) {
    v = *reinterpret_cast<const v4u_at1*>(p);
  } else {
    for (int k = 0; k < q - c; ++k) v[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
  }
  *reinterpret_cast<v4u8*>(dst + blockIdx.x * dld + c) = v;
}

constexpr int FEW8_COLS = 64;

template <int TA, int TB, bool WIDE, bool AROW, int B, int W>
hipError_t launch_tiles(const Scaled8& g, hipStream_t st) {
  using Tile = Tile8<TA, TB, WIDE, AROW, B, B, 2, W>;
  constexpr int SMEM = std::max(2 * Tile::BUF, Store<Tile>::BYTES);
  const long tiles = (long)((g.m + B - 1) / B) * ((g.n + B - 1) / B) * g.parts;
  auto kernel = scaled_tiles_kernel<Tile, B, B>;
  const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != hipSuccess) return e;
  kernel<<<(unsigned)tiles, Tile::THREADS, SMEM, st>>>(g);
  return hipGetLastError();
}

template <int TA, int TB, bool AROW>
hipError_t launch_few(const Scaled8& g, hipStream_t st) {
  const unsigned threads = FEW8_WAVES * 64;
  if (g.n <= 16)
    scaled_few_kernel<TA, TB, AROW, 1, 1><<<(g.m + 15) / 16, threads, 0, st>>>(g);
  else if (g.n <= 32)
    scaled_few_kernel<TA, TB, AROW, 1, 2><<<(g.m + 15) / 16, threads, 0, st>>>(g);
  else
    scaled_few_kernel<TA, TB, AROW, 1, 4><<<(g.m + 15) / 16, threads, 0, st>>>(g);
  return hipGetLastError();
}

template <int TA, int TB, bool AROW>
hipError_t launch_kind(const Scaled8& g, hipStream_t st) {
  if (g.n <= FEW8_COLS) return launch_few<TA, TB, AROW>(g, st);
  const long big = (long)((g.m + 255) / 256) * ((g.n + 255) / 256);
  const bool wide = g.ctype == OZGEMM_F32;
  hipError_t e;
  if (big >= 128)
    e = wide ? launch_tiles<TA, TB, true, AROW, 256, 4>(g, st) : launch_tiles<TA, TB, false, AROW, 256, 4>(g, st);
  else
    e = wide ? launch_tiles<TA, TB, true, AROW, 128, 2>(g, st) : launch_tiles<TA, TB, false, AROW, 128, 2>(g, st);
  if (e != hipSuccess || g.parts == 1) return e;
  join_parts_kernel<<<dim3(g.n, (g.m + 1023) / 1024), 256, 0, st>>>(g);
  return hipGetLastError();
}

template <int TA, int TB>
hipError_t launch_types(const Scaled8& g, hipStream_t st) {
  return g.A.shift == 0 ? launch_kind<TA, TB, true>(g, st) : launch_kind<TA, TB, false>(g, st);
}

}  // namespace

int scaled_parts(int ctype, int m, int n, int q) {
  (void)ctype;
  if (n <= FEW8_COLS) return 1;
  const long tiles = (long)((m + 127) / 128) * ((n + 127) / 128), blocks = (q + 127) / 128;
  if (tiles >= 256) return 1;
  return (int)std::max(1L, std::min(512 / tiles, blocks / 4));
}

bool scaled_fits(int m, int n, int parts) {
  if (n <= FEW8_COLS) return (m + 15) / 16 <= (1 << 23) - 1;  // blocks of 512 threads
  return (long)((m + 127) / 128) * ((n + 127) / 128) * parts <= (1L << 23) - 1;
}

hipError_t launch_scaled(const Scaled8& g, hipStream_t st) {
  constexpr int F = OZGEMM_E4M3, E = OZGEMM_E5M2;
  if (g.atype == F) return g.btype == F ? launch_types<F, F>(g, st) : launch_types<F, E>(g, st);
  return g.btype == F ? launch_types<E, F>(g, st) : launch_types<E, E>(g, st);
}

hipError_t launch_align_rows(const uint8_t* src, long ld, int rows, int q, uint8_t* dst, long dld, hipStream_t st) {
  const int pieces = (q + 4095) / 4096, some = ((1 << 24) - 1) / pieces;  // under 2^32 threads a launch
  for (int r = 0; r < rows; r += some)
    align_rows_kernel<<<dim3(std::min(some, rows - r), pieces), 256, 0, st>>>(src + r * ld, ld, q, dst + r * dld, dld);
  return hipGetLastError();
}

}  // namespace oz
