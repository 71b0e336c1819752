// Operands of the 16-bit products laid out K-contiguous in zero-padded
// planes: needed for FP32 operands, which become two half-precision slices,
// and for 16-bit operands whose rows do not lie on 16-byte boundaries.
//
// FP32 slices.  With 2^(e-1) <= max |x| < 2^e over a row, y = x 2^(15-e) is
// exact, hi = RN16(y) and lo = RN16(y - hi).  For y in [2^E, 2^(E+1)) half's
// step is 2^(E-10), so |y - hi| <= 2^(E-11); y - hi is exact in FP32, and lo
// is off by at most 2^(E-23): hi + lo is y up to 2^-23 relative (FP32 itself
// rounds to 2^-24) while |y| >= 2^-2, where lo's step is half's smallest,
// 2^-24; below that up to 2^-25 absolute, 2^-39 of the row's largest entry.
// hi hi, hi lo and lo hi give the product up to the dropped lo lo, at most
// 2^-22 of each term.  The rows' scaling is the library's own (a power of two
// per row of A and column of B); as there, a row holding Inf or NaN gets
// OZGEMM_EXP_NONFINITE and zero slices.
//
// The passes are bound by HBM: each plane is written once and each entry read
// once (twice where its row is K-strided or longer than a wavefront's
// registers hold: the maximum has to be known first).  In f32, 32768 rows of
// 2048 (268 MB read, as much written) take 107 us, 5.0 TB/s; 8192 rows 28.6 us.
// K-strided, 8192 x 2048: 28 us for the slices and 14 + 5 for the exponents.
#include "groups.h"
#include "pieces.h"
#include "products.h"
#include "tile16.h"

namespace oz {

namespace {

// frexp exponent of a float's |.| bit pattern; 0 for zero, the flag for Inf and NaN
__device__ __forceinline__ int exponent32(uint32_t b) {
  if (b == 0) return 0;
  if (b >= 0x7f800000u) return OZGEMM_EXP_NONFINITE;
  const int biased = (int)(b >> 23);
  return biased > 0 ? biased - 126 : (31 - __clz((int)b)) - 148;
}

// Four entries next to each other as 32-bit patterns (16-bit types travel as
// they are), zeros past `left`.
template <int TYPE>
__device__ __forceinline__ void load4(const void* src, long at, int left, uint32_t (&v)[4]) {
  if (TYPE == OZGEMM_F32) {
    const uint32_t* p = (const uint32_t*)src + at;
    if (left >= 4) {
      const v4u x = *reinterpret_cast<const v4u_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : 0;
  } else {
    const uint16_t* p = (const uint16_t*)src + at;
    if (left >= 4) {
      const v4s x = *reinterpret_cast<const v4s_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint16_t)x[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : 0;
  }
}

// hi in the low half, lo in the high one (16-bit types: the entry itself)
template <int TYPE>
__device__ __forceinline__ uint32_t slices_of(uint32_t bits, int e) {
  if (TYPE != OZGEMM_F32) return bits;
  if (e == OZGEMM_EXP_NONFINITE) return 0;
  const float y = __builtin_ldexpf(__builtin_bit_cast(float, bits), 15 - e);
  const _Float16 h = (_Float16)y;
  return __builtin_bit_cast(uint16_t, h) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)(y - (float)h)) << 16);
}

// The high halves and the low halves of four slices as two words each.
__device__ __forceinline__ uint2 lows(const uint32_t (&s)[4]) {
  return uint2{(s[0] & 0xffffu) | (s[1] << 16), (s[2] & 0xffffu) | (s[3] << 16)};
}
__device__ __forceinline__ uint2 highs(const uint32_t (&s)[4]) {
  return uint2{(s[0] >> 16) | (s[1] & 0xffff0000u), (s[2] >> 16) | (s[3] & 0xffff0000u)};
}

template <int TYPE>
__device__ __forceinline__ void put4(uint16_t* out, long plane, uint32_t (&v)[4], int e) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = slices_of<TYPE>(v[i], e);
  *reinterpret_cast<uint2*>(out) = lows(v);
  if (TYPE == OZGEMM_F32) *reinterpret_cast<uint2*>(out + plane) = highs(v);
}

// K-contiguous rows, a wavefront each: RUNS runs of four entries per lane are
// kept in registers between the row's maximum and its slices, so a row of up
// to 256 RUNS entries is read once; longer rows are read twice.
template <int TYPE, int RUNS>
__global__ __launch_bounds__(256) void slice_rows_kernel(const void* __restrict__ src, long ld, long sbatch, int rows,
                                                         long total, int K, uint16_t* __restrict__ dst, long dld,
                                                         long plane, int32_t* __restrict__ ex, long first) {
  const long row = (first + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= total) return;
  const long from = row / rows * sbatch + row % rows * ld;
  uint16_t* out = dst + row * dld;
  const int Kp = (K + 63) / 64 * 64;
  uint32_t v[RUNS][4];
  uint32_t mx = 0;
  const bool once = Kp <= 256 * RUNS;
  for (int k0 = 0; k0 < Kp; k0 += 256 * RUNS) {
#pragma unroll
    for (int i = 0; i < RUNS; ++i) load4<TYPE>(src, from + k0 + i * 256 + lane * 4, K - k0 - i * 256 - lane * 4, v[i]);
    if (TYPE != OZGEMM_F32) {
#pragma unroll
      for (int i = 0; i < RUNS; ++i)
        if (k0 + i * 256 + lane * 4 < Kp) put4<TYPE>(out + k0 + i * 256 + lane * 4, plane, v[i], 0);
    } else {
#pragma unroll
      for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = max(mx, v[i][j] & 0x7fffffffu);
    }
  }
  if (TYPE != OZGEMM_F32) return;
#pragma unroll
  for (int d = 32; d; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
  const int e = exponent32(mx);
  if (lane == 0) ex[row] = e;
  for (int k0 = 0; k0 < Kp; k0 += 256 * RUNS) {
    if (!once) {
#pragma unroll
      for (int i = 0; i < RUNS; ++i) load4<TYPE>(src, from + k0 + i * 256 + lane * 4, K - k0 - i * 256 - lane * 4, v[i]);
    }
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
      if (k0 + i * 256 + lane * 4 < Kp) put4<TYPE>(out + k0 + i * 256 + lane * 4, plane, v[i], e);
  }
}

// Tiles of TILE k: with offsets, of the ragged groups; else of `groups`
// matrices of K each.
struct KRange {
  int group;
  int k0, k1;   // within the source
  long dst_k;   // where k0 lands in a destination row
  int tile;     // the tile's place in its group
};

template <int TILE>
__device__ __forceinline__ KRange k_range(const int32_t* offsets, int groups, int K, long idx) {
  if (offsets == nullptr) {
    const int per = (K + TILE - 1) / TILE;
    const int b = (int)(idx / per), t = (int)(idx % per);
    return KRange{b, t * TILE, min(K, (t + 1) * TILE), (long)t * TILE, t};
  }
  const GroupTile g = find_group_tile(offsets, groups, K, TILE, (int)idx);
  return KRange{g.group, g.begin, min(g.end, g.begin + TILE), idx * TILE, g.tile};
}

// Bits of the largest |entry| of every column r of a tile of CHUNK k, one
// block per 256 columns: part[tile][r].
constexpr int CHUNK = 64;

__global__ __launch_bounds__(256) void column_max_kernel(const float* __restrict__ src, long ld, long sbatch,
                                                         int rows, int K, const int32_t* __restrict__ offsets,
                                                         int groups, uint32_t* __restrict__ part, long first) {
  const long idx = first + blockIdx.x;
  const KRange g = k_range<CHUNK>(offsets, groups, K, idx);
  if (g.group < 0) return;
  const int lane = threadIdx.x & 63, r = blockIdx.y * 256 + lane * 4;
  const long base = offsets ? 0 : g.group * sbatch;
  uint32_t mx[4] = {0, 0, 0, 0};
  if (r < rows) {
    // eight loads in flight; a k past the end reads the last one again
    for (int k = g.k0 + (threadIdx.x >> 6); k < g.k1; k += 32) {
      uint32_t v[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) load4<OZGEMM_F32>(src, base + (long)min(k + 4 * i, g.k1 - 1) * ld + r, rows - r, v[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = max(mx[j], v[i][j] & 0x7fffffffu);
    }
  }
  __shared__ uint32_t s[4][256];
#pragma unroll
  for (int j = 0; j < 4; ++j) s[threadIdx.x >> 6][lane * 4 + j] = mx[j];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < rows)
    part[idx * rows + c] = max(max(s[0][threadIdx.x], s[1][threadIdx.x]), max(s[2][threadIdx.x], s[3][threadIdx.x]));
}

// The exponents of 64 columns of one group from its chunks' maxima.
__global__ __launch_bounds__(256) void column_exponents_kernel(const uint32_t* __restrict__ part, int rows, int K,
                                                               const int32_t* __restrict__ offsets, int groups,
                                                               int32_t* __restrict__ ex) {
  const int e = blockIdx.x, lane = threadIdx.x & 63, r = blockIdx.y * 64 + lane;
  int count = (K + CHUNK - 1) / CHUNK, first = e * count;
  if (offsets) {
    const GroupTile g = group_at(offsets, groups, K, CHUNK, e);
    first = g.first;
    count = (g.end - g.begin + CHUNK - 1) / CHUNK;
  }
  uint32_t mx = 0;
  if (r < rows) {
    for (int c = threadIdx.x >> 6; c < count; c += 32) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(long)(first + min(c + 4 * i, count - 1)) * rows + r];
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = max(mx, v[i]);
    }
  }
  __shared__ uint32_t s[4][64];
  s[threadIdx.x >> 6][lane] = mx;
  __syncthreads();
  if (threadIdx.x < 64 && r < rows) ex[(long)e * rows + r] = exponent32(max(max(s[0][lane], s[1][lane]), max(s[2][lane], s[3][lane])));
}

// A 64 x 64 tile of K-strided entries, cut into slices and transposed through
// LDS.
template <int TYPE>
__global__ __launch_bounds__(256) void slice_cols_kernel(const void* __restrict__ src, long ld, long sbatch, int rows,
                                                         int K, const int32_t* __restrict__ offsets, int groups,
                                                         uint16_t* __restrict__ dst, long dld, long plane,
                                                         const int32_t* __restrict__ ex, long first) {
  const KRange g = k_range<64>(offsets, groups, K, first + blockIdx.x);
  if (g.group < 0) return;
  __shared__ uint32_t tile[64][65];
  __shared__ int32_t es[64];
  const int r0 = blockIdx.y * 64;
  const long from = offsets ? 0 : g.group * sbatch;
  const int rr = (threadIdx.x & 15) * 4, kk = threadIdx.x >> 4;
  uint32_t v[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = g.k0 + kk + 16 * i;
    load4<TYPE>(src, from + (long)k * ld + r0 + rr, k < g.k1 ? rows - r0 - rr : 0, v[i]);
  }
  if (TYPE == OZGEMM_F32) {
    if (threadIdx.x < 64) es[threadIdx.x] = r0 + (int)threadIdx.x < rows ? ex[(long)g.group * rows + r0 + threadIdx.x] : 0;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tile[kk + 16 * i][rr + j] = slices_of<TYPE>(v[i][j], TYPE == OZGEMM_F32 ? es[rr + j] : 0);
  __syncthreads();
  uint16_t* base = dst + (offsets ? 0 : (long)g.group * rows * dld) + g.dst_k;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = half * 256 + threadIdx.x, r = i >> 3, k = (i & 7) * 8;
    if (r0 + r >= rows) continue;
    uint32_t a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = tile[k + j][r];
      b[j] = tile[k + 4 + j][r];
    }
    uint16_t* out = base + (long)(r0 + r) * dld + k;
    const uint2 la = lows(a), lb = lows(b);
    *reinterpret_cast<uint4*>(out) = uint4{la.x, la.y, lb.x, lb.y};
    if (TYPE == OZGEMM_F32) {
      const uint2 ha = highs(a), hb = highs(b);
      *reinterpret_cast<uint4*>(out + plane) = uint4{ha.x, ha.y, hb.x, hb.y};
    }
  }
}

long k_tiles(const int32_t* offsets, long K, long groups, long tile) {
  return offsets ? group_tiles_max(K, groups, tile) : (K + tile - 1) / tile * groups;
}

hipError_t slice_cols(int type, const void* src, long ld, long sbatch, int rows, int K, const int32_t* offsets,
                      int groups, uint16_t* dst, long dld, long plane, int32_t* ex, uint32_t* part, hipStream_t st) {
  if (rows < 1 || K < 1 || groups < 1) return hipSuccess;
  const long tiles = k_tiles(offsets, K, groups, 64);
  const unsigned row_tiles = (unsigned)((rows + 63) / 64);
  if (type == OZGEMM_F32) {
    in_pieces(k_tiles(offsets, K, groups, CHUNK), [&](long first, unsigned count) {
      hipLaunchKernelGGL(column_max_kernel, dim3(count, (unsigned)((rows + 255) / 256)), dim3(256), 0, st,
                         (const float*)src, ld, sbatch, rows, K, offsets, groups, part, first);
    });
    hipLaunchKernelGGL(column_exponents_kernel, dim3(groups, row_tiles), dim3(256), 0, st, part, rows, K, offsets,
                       groups, ex);
  }
  in_pieces(tiles, [&](long first, unsigned count) {
    if (type == OZGEMM_F32)
      hipLaunchKernelGGL(slice_cols_kernel<OZGEMM_F32>, dim3(count, row_tiles), dim3(256), 0, st, src, ld, sbatch, rows,
                         K, offsets, groups, dst, dld, plane, ex, first);
    else
      hipLaunchKernelGGL(slice_cols_kernel<OZGEMM_F16>, dim3(count, row_tiles), dim3(256), 0, st, src, ld, sbatch, rows,
                         K, offsets, groups, dst, dld, plane, ex, first);
  });
  return hipGetLastError();
}

template <int TYPE, int RUNS>
hipError_t slice_rows(const void* src, long ld, long sbatch, int rows, long total, int K, uint16_t* dst, long dld,
                      long plane, int32_t* ex, hipStream_t st) {
  in_pieces((total + 3) / 4, [&](long first, unsigned count) {
    hipLaunchKernelGGL((slice_rows_kernel<TYPE, RUNS>), dim3(count), dim3(256), 0, st, src, ld, sbatch, rows, total, K,
                       dst, dld, plane, ex, first);
  });
  return hipGetLastError();
}

}  // namespace

size_t slice_part_bytes(int rows, long K, int groups, bool ragged) {
  return (size_t)k_tiles(ragged ? (const int32_t*)1 : nullptr, K, groups, CHUNK) * rows * 4;
}

hipError_t launch_slice_rows(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st) {
  if (rows < 1 || batches < 1 || K < 1) return hipSuccess;
  const long n = (long)rows * batches;
  if (type != OZGEMM_F32) return slice_rows<OZGEMM_F16, 4>(src, ld, sbatch, rows, n, K, dst, dld, plane, ex, st);
  if (K <= 1024) return slice_rows<OZGEMM_F32, 4>(src, ld, sbatch, rows, n, K, dst, dld, plane, ex, st);
  if (K <= 2048) return slice_rows<OZGEMM_F32, 8>(src, ld, sbatch, rows, n, K, dst, dld, plane, ex, st);
  return slice_rows<OZGEMM_F32, 16>(src, ld, sbatch, rows, n, K, dst, dld, plane, ex, st);
}

hipError_t launch_slice_cols(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, uint32_t* part, hipStream_t st) {
  return slice_cols(type, src, ld, sbatch, rows, K, nullptr, batches, dst, dld, plane, ex, part, st);
}

hipError_t launch_slice_groups(int type, const void* src, long ld, int rows, int n, const int32_t* offsets,
                               int groups, uint16_t* dst, long dld, long plane, int32_t* ex, uint32_t* part,
                               hipStream_t st) {
  return slice_cols(type, src, ld, 0, rows, n, offsets, groups, dst, dld, plane, ex, part, st);
}

}  // namespace oz
