// The norm over all entries of many arrays, and their scaling by it.
//
//   N = sqrt(sum over the arrays of sum g^2),  o = g min(1, most / (N + eps))
//
// The arrays' addresses and sizes travel in the launch's arguments, TABLE
// arrays a launch, so nothing is copied from the host.  An array is cut into
// chunks; a block sums one in FP64 (squares of the 16- and 32-bit types are
// exact there) into a place of its own, and one block adds those up in a
// fixed order.
//
// Bound by HBM: 48 arrays of BF16, 957 MB together, 196 us for the norm (4.9 TB/s) and
// 347 us for the scaling (5.5 TB/s); nothing can be scaled before all of it is read, and
// the caches hold a quarter of it at best: going through the arrays backwards the second time
// gained nothing.  40 small ones: 5.8, 1.8 and 8.6 us in three launches.
#include <algorithm>
#include <vector>

#include "block8.h"
#include "products.h"

namespace oz {
namespace {

constexpr int TABLE = 96;            // 24 bytes each: a launch's arguments go up to 4 KiB
constexpr long CHUNK_BYTES = 65536;  // of one block: 16 loads of 16 bytes per thread

struct Table {
  const void* in[TABLE];
  void* out[TABLE];
  long size[TABLE];
  int first[TABLE + 1];  // chunks before an array's
  uint8_t type[TABLE];
  int count;
};

int chunk_entries(int type) { return (int)(CHUNK_BYTES / elem_bytes(type)); }

// The array of the block's chunk, its chunk there.
__device__ __forceinline__ int find(const Table& t, int& chunk) {
  int lo = 0, hi = t.count;  // first[lo] <= block < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= (int)blockIdx.x)
      lo = mid;
    else
      hi = mid;
  }
  chunk = blockIdx.x - t.first[lo];
  return lo;
}

template <int TYPE>
__device__ __forceinline__ double square_sum(const void* p, long size, int chunk) {
  constexpr int PER = CHUNK_BYTES / Entry<TYPE>::BYTES, STEP = 256 * 8;
  const long at = (long)chunk * PER;
  const int left = (int)min((long)PER, size - at);
  double s = 0;
#pragma unroll 4
  for (int k = threadIdx.x * 8; k < left; k += STEP) {
    Raw8<TYPE> v;
    v.load(p, at + k, left - k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double x = (double)v.get(i);
      s = __builtin_fma(x, x, s);
    }
  }
  return s;
}

__device__ __forceinline__ double square_sum64(const double* p, long size, int chunk) {
  constexpr int PER = CHUNK_BYTES / 8;
  const long at = (long)chunk * PER;
  const int left = (int)min((long)PER, size - at);
  double s = 0;
#pragma unroll 4
  for (int k = threadIdx.x; k < left; k += 256) s = __builtin_fma(p[at + k], p[at + k], s);
  return s;
}

template <int THREADS>
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double meet[THREADS / 64];
  s = sum64(s);
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = s;
  __syncthreads();
  s = meet[0];
#pragma unroll
  for (int k = 1; k < THREADS / 64; ++k) s += meet[k];
  return s;
}

__global__ __launch_bounds__(256) void square_sums_kernel(Table t, double* sums) {
  int chunk;
  const int a = find(t, chunk);
  const int type = t.type[a];
  double s;
  if (type == OZGEMM_F32)
    s = square_sum<OZGEMM_F32>(t.in[a], t.size[a], chunk);
  else if (type == OZGEMM_BF16)
    s = square_sum<OZGEMM_BF16>(t.in[a], t.size[a], chunk);
  else if (type == OZGEMM_F16)
    s = square_sum<OZGEMM_F16>(t.in[a], t.size[a], chunk);
  else
    s = square_sum64((const double*)t.in[a], t.size[a], chunk);
  s = block_sum<256>(s);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void join_norm_kernel(const double* sums, long n, double* norm) {
  double s = 0;
#pragma unroll 8
  for (long k = threadIdx.x; k < n; k += 1024) s += sums[k];
  s = block_sum<1024>(s);
  if (threadIdx.x == 0) *norm = sqrt(s);
}

// A factor's 24 bits for entries of up to 32 bits: x times it is ((x step) f) step, where
// the step is 1, or 2^-100 for factors below that, which FP32 holds in fewer bits or not at all.
struct Factor {
  float f, step;
  __device__ __forceinline__ explicit Factor(double v)
      : f((float)(v < 0x1p-100 ? v * 0x1p200 : v)), step(v < 0x1p-100 ? 0x1p-100f : 1.f) {}
  __device__ __forceinline__ float times(float x) const { return x * step * f * step; }
};

template <int TYPE>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, long size, int chunk, Factor f) {
  constexpr int PER = CHUNK_BYTES / Entry<TYPE>::BYTES, STEP = 256 * 8;
  const long at = (long)chunk * PER;
  const int left = (int)min((long)PER, size - at);
#pragma unroll 4
  for (int k = threadIdx.x * 8; k < left; k += STEP) {
    Raw8<TYPE> v;
    v.load(in, at + k, left - k);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f.times(v.get(i));
    v.set(x);
    v.store(out, at + k, left - k);
  }
}

__global__ __launch_bounds__(256) void scale_kernel(Table t, const double* norm, double most, double eps) {
  int chunk;
  const int a = find(t, chunk);
  // NaN stays: a norm that is none makes every entry NaN
  const double q = most / (*norm + eps), f = q > 1.0 ? 1.0 : q;
  if (f == 1.0 && t.in[a] == t.out[a]) return;  // x 1 is x
  const int type = t.type[a];
  if (type == OZGEMM_F32) {
    scale_chunk<OZGEMM_F32>(t.in[a], t.out[a], t.size[a], chunk, Factor(f));
  } else if (type == OZGEMM_BF16) {
    scale_chunk<OZGEMM_BF16>(t.in[a], t.out[a], t.size[a], chunk, Factor(f));
  } else if (type == OZGEMM_F16) {
    scale_chunk<OZGEMM_F16>(t.in[a], t.out[a], t.size[a], chunk, Factor(f));
  } else {
    constexpr int PER = CHUNK_BYTES / 8;
    const double* p = (const double*)t.in[a];
    double* o = (double*)t.out[a];
    const long at = (long)chunk * PER;
    const int left = (int)min((long)PER, t.size[a] - at);
    for (int k = threadIdx.x; k < left; k += 256) o[at + k] = p[at + k] * f;
  }
}

long chunks_of(int type, long long size) {
  const long per = chunk_entries(type);
  return (long)((size + per - 1) / per);
}

// Calls f(table, chunks, chunks before) for the arrays with entries, at most
// TABLE of them and 2^24 - 1 chunks (2^32 threads) a launch.  An array with
// more is handed over in parts.
template <class F>
hipError_t in_tables(int count, const int* types, const void* const* in, void* const* out, const long long* sizes,
                     F f) {
  constexpr long CHUNKS_MAX = (1L << 24) - 1;
  Table t{};
  long before = 0, now = 0;
  auto flush = [&]() {
    t.first[t.count] = (int)now;
    f(t, now, before);
    before += now;
    now = 0;
    t.count = 0;
    return hipGetLastError();
  };
  for (int k = 0; k < count; ++k) {
    const long per = chunk_entries(types[k]);
    const size_t bytes = elem_bytes(types[k]);
    for (long done = 0; done < sizes[k];) {
      if (t.count == TABLE || now == CHUNKS_MAX) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      const long some = std::min((long)(sizes[k] - done), (CHUNKS_MAX - now) * per);
      t.in[t.count] = (const char*)in[k] + done * bytes;
      t.out[t.count] = out ? (char*)out[k] + done * bytes : nullptr;
      t.size[t.count] = some;
      t.type[t.count] = (uint8_t)types[k];
      t.first[t.count++] = (int)now;
      now += chunks_of(types[k], some);
      done += some;
    }
  }
  return t.count > 0 ? flush() : hipSuccess;
}

bool known_grad(int type) {
  return type == OZGEMM_F64 || type == OZGEMM_F32 || type == OZGEMM_BF16 || type == OZGEMM_F16;
}

// The arguments that both calls share: 0, or which is wrong.
int check_arrays(int count, const int* types, const void* const* in, const long long* sizes) {
  if (count < 0 || count > OZGEMM_ARRAYS_MAX) return -1;
  if (count == 0) return 0;
  if (types == nullptr) return -2;
  if (in == nullptr) return -3;
  if (sizes == nullptr) return -4;
  for (int k = 0; k < count; ++k) {
    if (!known_grad(types[k])) return -2;
    if (sizes[k] < 0 || sizes[k] > OZGEMM_ARRAY_MAX) return -4;
    if (in[k] == nullptr && sizes[k] > 0) return -3;
  }
  return 0;
}

size_t sums_bytes(int count, const int* types, const long long* sizes) {
  size_t chunks = 0;
  for (int k = 0; k < count; ++k) chunks += chunks_of(types[k], sizes[k]);
  return up(std::max<size_t>(chunks, 1) * sizeof(double), 256);
}

struct Span {
  const char *from, *to;
};

// Whether any of `written` shares memory with another or with any of `read`.
bool any_overlap(std::vector<Span>& written, std::vector<Span>& read) {
  const auto before = [](const Span& a, const Span& b) { return a.from < b.from; };
  std::sort(written.begin(), written.end(), before);
  std::sort(read.begin(), read.end(), before);
  for (size_t k = 1; k < written.size(); ++k)
    if (written[k].from < written[k - 1].to) return true;
  size_t w = 0;  // the first that ends behind the span's beginning
  for (const Span& r : read) {
    while (w < written.size() && written[w].to <= r.from) ++w;
    if (w < written.size() && written[w].from < r.to) return true;
  }
  return false;
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozgemm_gradient_norm_workspace_bytes(int count, const int* types, const long long* sizes) {
  if (count < 0 || count > OZGEMM_ARRAYS_MAX || (count > 0 && (types == nullptr || sizes == nullptr))) return 0;
  for (int k = 0; k < count; ++k)
    if (!known_grad(types[k]) || sizes[k] < 0 || sizes[k] > OZGEMM_ARRAY_MAX) return 0;
  return sums_bytes(count, types, sizes);
}

int ozgemm_gradient_norm(int count, const int* types, const void* const* in, const long long* sizes, double* norm,
                         void* workspace, size_t workspace_bytes, void* hip_stream) {
  const int bad = check_arrays(count, types, in, sizes);
  if (bad != 0) return bad;
  if (norm == nullptr) return -5;
  for (int k = 0; k < count; ++k)
    if (overlap(norm, sizeof(double), in[k], (size_t)sizes[k] * elem_bytes(types[k]))) return -5;
  if (workspace == nullptr || ((uintptr_t)workspace & 255)) return -6;
  if (workspace_bytes < sums_bytes(count, types, sizes)) return OZGEMM_WORKSPACE_TOO_SMALL;
  hipStream_t st = (hipStream_t)hip_stream;
  double* sums = (double*)workspace;
  long total = 0;
  hipError_t e = in_tables(count, types, in, nullptr, sizes, [&](const Table& t, long chunks, long before) {
    square_sums_kernel<<<(unsigned)chunks, 256, 0, st>>>(t, sums + before);
    total = before + chunks;
  });
  if (e == hipSuccess) {
    join_norm_kernel<<<1, 1024, 0, st>>>(sums, total, norm);
    e = hipGetLastError();
  }
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}

int ozgemm_clip_gradients(int count, const int* types, const void* const* in, const long long* sizes,
                          void* const* out, const double* norm, double most, double eps, void* hip_stream) {
  const int bad = check_arrays(count, types, in, sizes);
  if (bad != 0) return bad;
  if (count > 0 && out == nullptr) return -5;
  for (int k = 0; k < count; ++k)
    if (out[k] == nullptr && sizes[k] > 0) return -5;
  if (norm == nullptr) return -6;
  if (!(most >= 0.0)) return -7;
  if (!(eps >= 0.0)) return -8;
  // Blocks write while others read: what is written is nobody else's, but for
  // the array that it comes from.  (No exception may leave this call.)
  try {
    std::vector<Span> written, read;
    written.reserve((size_t)count);
    read.reserve((size_t)count + 1);
    read.push_back({(const char*)norm, (const char*)norm + sizeof(double)});
    for (int k = 0; k < count; ++k) {
      if (sizes[k] == 0) continue;
      const size_t bytes = (size_t)sizes[k] * elem_bytes(types[k]);
      written.push_back({(const char*)out[k], (const char*)out[k] + bytes});
      if (in[k] != out[k]) read.push_back({(const char*)in[k], (const char*)in[k] + bytes});
    }
    if (any_overlap(written, read)) return -5;
  } catch (...) {
    return OZGEMM_RANGE;
  }
  hipStream_t st = (hipStream_t)hip_stream;
  const hipError_t e = in_tables(count, types, in, out, sizes, [&](const Table& t, long chunks, long) {
    scale_kernel<<<(unsigned)chunks, 256, 0, st>>>(t, norm, most, eps);
  });
  return e == hipSuccess ? OZGEMM_OK : record_hip_error(e);
}

}  // extern "C"
