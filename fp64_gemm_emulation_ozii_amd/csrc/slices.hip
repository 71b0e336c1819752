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
// The passes are bound by HBM: each entry is read once (the row maxima of
// K-contiguous rows twice, the second time from L2) and each plane written
// once.
#include "groups.h"
#include "products.h"

namespace oz {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// frexp exponent of a float's |.| bit pattern; 0 for zero, the flag for Inf and NaN
__device__ __forceinline__ int exponent32(uint32_t b) {
  if (b == 0) return 0;
  if (b >= 0x7f800000u) return OZGEMM_EXP_NONFINITE;
  const int biased = (int)(b >> 23);
  return biased > 0 ? biased - 126 : (31 - __clz((int)b)) - 148;
}

// bits of one entry, widened to 32 (16-bit types travel as they are)
template <int TYPE>
__device__ __forceinline__ uint32_t load_bits(const void* src, long at) {
  return TYPE == OZGEMM_F32 ? ((const uint32_t*)src)[at] : ((const uint16_t*)src)[at];
}

template <int TYPE>
__device__ __forceinline__ void slices_of(uint32_t bits, int e, uint16_t& hi, uint16_t& lo) {
  if (TYPE != OZGEMM_F32) {
    hi = (uint16_t)bits;
    lo = 0;
    return;
  }
  if (e == OZGEMM_EXP_NONFINITE) {
    hi = lo = 0;
    return;
  }
  const float y = __builtin_ldexpf(__builtin_bit_cast(float, bits), 15 - e);
  const _Float16 h = (_Float16)y;
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, (_Float16)(y - (float)h));
}

// One block per row: its maximum, then its slices.
template <int TYPE>
__global__ __launch_bounds__(256) void slice_rows_kernel(const void* __restrict__ src, long ld, long sbatch, int rows,
                                                         int K, uint16_t* __restrict__ dst, long dld, long plane,
                                                         int32_t* __restrict__ ex) {
  const long row = blockIdx.x;
  const long from = row / rows * sbatch + row % rows * ld;
  uint16_t* out = dst + row * dld;
  const int Kp = (K + 63) / 64 * 64;
  int e = 0;
  if (TYPE == OZGEMM_F32) {
    uint32_t mx = 0;
    for (int k = threadIdx.x; k < K; k += 256) mx = max(mx, load_bits<TYPE>(src, from + k) & 0x7fffffffu);
    __shared__ uint32_t part[4];
#pragma unroll
    for (int d = 32; d; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mx;
    __syncthreads();
    e = exponent32(max(max(part[0], part[1]), max(part[2], part[3])));
    if (threadIdx.x == 0) ex[row] = e;
  }
  for (int k = threadIdx.x * 2; k < Kp; k += 512) {
    uint16_t h0 = 0, l0 = 0, h1 = 0, l1 = 0;
    if (k < K) slices_of<TYPE>(load_bits<TYPE>(src, from + k), e, h0, l0);
    if (k + 1 < K) slices_of<TYPE>(load_bits<TYPE>(src, from + k + 1), e, h1, l1);
    *reinterpret_cast<uint32_t*>(out + k) = h0 | ((uint32_t)h1 << 16);
    if (TYPE == OZGEMM_F32) *reinterpret_cast<uint32_t*>(out + plane + k) = l0 | ((uint32_t)l1 << 16);
  }
}

__global__ __launch_bounds__(256) void fill_exponents_kernel(int32_t* __restrict__ ex, long n) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) ex[i] = 0;
}

// The columns' maxima bits into ex (as unsigned integers; zero before), one
// block per 64 rows r and CHUNK k.  With offsets, the k of group e; else
// batch e's.
constexpr int CHUNK = 256;

struct KRange {
  int group;
  int k0, k1;   // within the source
  long dst_k;   // where k0 lands in a destination row
};

template <int TILE>
__device__ __forceinline__ KRange k_range(const int32_t* offsets, int groups, int K, int idx) {
  if (offsets == nullptr) {
    const int per = (K + TILE - 1) / TILE;
    const int b = idx / per, t = idx % per;
    return KRange{b, t * TILE, min(K, (t + 1) * TILE), (long)t * TILE};
  }
  const GroupTile g = find_group_tile(offsets, groups, K, TILE, idx);
  return KRange{g.group, g.begin, min(g.end, g.begin + TILE), (long)idx * TILE};
}

__global__ __launch_bounds__(256) void column_max_kernel(const float* __restrict__ src, long ld, long sbatch,
                                                         int rows, int K, const int32_t* __restrict__ offsets,
                                                         int groups, uint32_t* __restrict__ ex) {
  const KRange g = k_range<CHUNK>(offsets, groups, K, blockIdx.x);
  if (g.group < 0) return;
  const int r = blockIdx.y * 64 + (threadIdx.x & 63);
  const uint32_t* p = (const uint32_t*)src + (offsets ? 0 : g.group * sbatch);
  uint32_t mx = 0;
  if (r < rows)
    for (int k = g.k0 + (threadIdx.x >> 6); k < g.k1; k += 4) mx = max(mx, p[(long)k * ld + r] & 0x7fffffffu);
  __shared__ uint32_t part[4][64];
  part[threadIdx.x >> 6][threadIdx.x & 63] = mx;
  __syncthreads();
  if (threadIdx.x < 64 && r < rows) {
    mx = max(max(part[0][threadIdx.x], part[1][threadIdx.x]), max(part[2][threadIdx.x], part[3][threadIdx.x]));
    if (mx) atomicMax(ex + (long)g.group * rows + r, mx);  // a maximum: the order does not matter
  }
}

__global__ __launch_bounds__(256) void exponents_kernel(int32_t* __restrict__ ex, long n) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) ex[i] = exponent32((uint32_t)ex[i]);
}

// A 64 x 64 tile of K-strided entries, transposed through LDS.
template <int TYPE>
__global__ __launch_bounds__(256) void slice_cols_kernel(const void* __restrict__ src, long ld, long sbatch, int rows,
                                                         int K, const int32_t* __restrict__ offsets, int groups,
                                                         uint16_t* __restrict__ dst, long dld, long plane,
                                                         const int32_t* __restrict__ ex) {
  const KRange g = k_range<64>(offsets, groups, K, blockIdx.x);
  if (g.group < 0) return;
  __shared__ uint32_t tile[64][65];
  const int r0 = blockIdx.y * 64;
  const long from = offsets ? 0 : g.group * sbatch;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int k = i >> 6, r = i & 63;
    tile[k][r] = g.k0 + k < g.k1 && r0 + r < rows ? load_bits<TYPE>(src, from + (long)(g.k0 + k) * ld + r0 + r) : 0;
  }
  __syncthreads();
  uint16_t* base = dst + (offsets ? 0 : (long)g.group * rows * dld) + g.dst_k;
  for (int i = threadIdx.x; i < 64 * 32; i += 256) {
    const int r = i >> 5, k = (i & 31) * 2;
    if (r0 + r < rows) {
      const int e = TYPE == OZGEMM_F32 ? ex[(long)g.group * rows + r0 + r] : 0;
      uint16_t h0, l0, h1, l1;
      slices_of<TYPE>(tile[k][r], e, h0, l0);
      slices_of<TYPE>(tile[k + 1][r], e, h1, l1);
      uint16_t* out = base + (long)(r0 + r) * dld + k;
      *reinterpret_cast<uint32_t*>(out) = h0 | ((uint32_t)h1 << 16);
      if (TYPE == OZGEMM_F32) *reinterpret_cast<uint32_t*>(out + plane) = l0 | ((uint32_t)l1 << 16);
    }
  }
}

hipError_t slice_cols(int type, const void* src, long ld, long sbatch, int rows, int K, const int32_t* offsets,
                      int groups, uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st) {
  if (rows < 1 || K < 1 || groups < 1) return hipSuccess;
  const unsigned rt = (unsigned)((rows + 63) / 64);
  const auto tiles = [&](long tile) {
    return offsets ? group_tiles_max(K, groups, tile) : (K + tile - 1) / tile * groups;
  };
  if (tiles(64) > 0x7fffffffL || rt > 65535) return hipErrorInvalidValue;
  if (type == OZGEMM_F32) {
    const long n = (long)groups * rows;
    const dim3 g1((unsigned)((n + 255) / 256));
    hipLaunchKernelGGL(fill_exponents_kernel, g1, dim3(256), 0, st, ex, n);
    hipLaunchKernelGGL(column_max_kernel, dim3((unsigned)tiles(CHUNK), rt), dim3(256), 0, st, (const float*)src, ld,
                       sbatch, rows, K, offsets, groups, (uint32_t*)ex);
    hipLaunchKernelGGL(exponents_kernel, g1, dim3(256), 0, st, ex, n);
    hipLaunchKernelGGL(slice_cols_kernel<OZGEMM_F32>, dim3((unsigned)tiles(64), rt), dim3(256), 0, st, src, ld,
                       sbatch, rows, K, offsets, groups, dst, dld, plane, ex);
  } else {
    hipLaunchKernelGGL(slice_cols_kernel<OZGEMM_F16>, dim3((unsigned)tiles(64), rt), dim3(256), 0, st, src, ld,
                       sbatch, rows, K, offsets, groups, dst, dld, plane, ex);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_slice_rows(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st) {
  if (rows < 1 || batches < 1 || K < 1) return hipSuccess;
  const long n = (long)rows * batches;
  if (n > 0x7fffffffL) return hipErrorInvalidValue;
  if (type == OZGEMM_F32)
    hipLaunchKernelGGL(slice_rows_kernel<OZGEMM_F32>, dim3((unsigned)n), dim3(256), 0, st, src, ld, sbatch, rows, K,
                       dst, dld, plane, ex);
  else
    hipLaunchKernelGGL(slice_rows_kernel<OZGEMM_F16>, dim3((unsigned)n), dim3(256), 0, st, src, ld, sbatch, rows, K,
                       dst, dld, plane, ex);
  return hipGetLastError();
}

hipError_t launch_slice_cols(int type, const void* src, long ld, long sbatch, int batches, int rows, int K,
                             uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st) {
  return slice_cols(type, src, ld, sbatch, rows, K, nullptr, batches, dst, dld, plane, ex, st);
}

hipError_t launch_slice_groups(int type, const void* src, long ld, int rows, int n, const int32_t* offsets,
                               int groups, uint16_t* dst, long dld, long plane, int32_t* ex, hipStream_t st) {
  return slice_cols(type, src, ld, 0, rows, n, offsets, groups, dst, dld, plane, ex, st);
}

}  // namespace oz
