// One output tile of a product of 16-bit operands on gfx950 matrix cores:
//   acc[i][j] = sum over k of A[i][k] B[j][k]
// with the accumulators in FP32.  Shared by the grouped products
// (gemm16.hip) and the Newton-Schulz steps (ortho.hip).
//
// An operand lies "K-contiguous" (row i at i ld, its entries next to each
// other) or "K-strided" (entry (i, k) at k ld + i).  K slices of 64 entries
// go from HBM straight into LDS (16 bytes per lane) through two buffers, in
// the operand's own order; a K-strided tile is transposed on its way from
// LDS into registers (ds_read_b64_tr_b16: 16 lanes read 4 x 16 entries and
// each receives a column of 4).  The loads carry a range check: what lies
// past the operand's end arrives as zero, and entries past the inner
// dimension of a K-contiguous row are sent past the end, so ragged edges
// cost no branch and never meet their neighbours' values.
//
// An operand may come as two slices (hi + lo, see slices.hip); three slice
// products lo hi, hi lo, hi hi (smallest first) are then walked as one long
// K loop into the same accumulators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oz {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

struct Half {
  static __device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};
struct Bfloat {
  static __device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                   0);
  }
};

// Where one operand's tile begins and what may be read from there on.
struct Source16 {
  const uint16_t* base;  // first entry of the tile at k = 0
  long plane;            // distance to the second slice
  int ld;
  int rows;  // K-contiguous: rows from `base` on that exist (more than a tile has: as many as it has)
  int last;  // entries that may be read of the last row (K-contiguous) or of the last k (K-strided) from `base` on
};

constexpr int BK16 = 64;  // K entries per slice: 128 bytes of a K-contiguous row

// Largest leading dimension the 32-bit offsets within a tile allow:
// 256 rows of 2 ld bytes stay below 2^30.
constexpr long LD16_MAX = 1L << 21;

template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// This wave's LDS reads are done and its loads into LDS have landed; then
// every wave's.
__device__ __forceinline__ void slice_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <class T, int BM, int BN, int WM, int WN, bool AKS, bool BKS>
struct Tile16 {
  static constexpr int NW = WM * WN, WAVES_N = WN;
  static constexpr int THREADS = NW * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int A_BYTES = BM * BK16 * 2, B_BYTES = BN * BK16 * 2;
  static constexpr int BUF = A_BYTES + B_BYTES;
  static constexpr int SMEM = 2 * BUF;
  static constexpr int A_LOADS = A_BYTES / 1024 / NW, B_LOADS = B_BYTES / 1024 / NW;
  static_assert(A_LOADS * NW * 1024 == A_BYTES && B_LOADS * NW * 1024 == B_BYTES, "whole wave loads");
  static_assert(FM * WM * 16 == BM && FN * WN * 16 == BN, "whole matrix-core tiles");

  // K-contiguous rows of 128 bytes: 16-byte chunk c of row r sits at chunk
  // c ^ swz(r), so that the 16 rows of an operand read fall in different
  // 16-byte bank slots (as in the int8 product).
  static __device__ __forceinline__ int swz(int row) { return ((row >> 1) ^ (row << 2)) & 7; }

  // K-strided rows of ROWS 16-bit entries (one row per k): 32-byte piece p of
  // row k sits at piece p ^ kswz(k).  A transposing read takes 8 rows k (0..3
  // and 8..11 past a multiple of 4) of one piece per 32 lanes; kswz sends
  // them to 8 different bank slots.
  template <int ROWS>
  static __device__ __forceinline__ int kswz(int k) {
    return ROWS >= 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
  }

  // The loads of one operand.  Within a slice, wave load number blk fills
  // LDS bytes [blk 1024, + 1024).
  template <int ROWS, bool KS, int LOADS>
  struct Loader {
    const char* p;   // the slice to load: its base,
    int records;     // the bytes that may be read from there
    int ld;
    int off[2];      // lane's byte offset in an even and an odd load (K-contiguous)
    int kin[2];      // lane's first k within the slice
    int base[2];     // off, or past the end for a lane whose k lies past the inner dimension
    int last, rows;
    int lane, wave;

    __device__ __forceinline__ void init(const Source16& s, int lane_, int wave_) {
      ld = s.ld;
      last = s.last;
      rows = min(s.rows, ROWS);
      lane = lane_;
      wave = wave_;
      if (!KS) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = lane >> 3, c = (lane & 7) ^ swz(e * 8 + r);
          off[e] = (r * ld + c * 8) * 2;
          kin[e] = c * 8;
        }
      }
    }

    // The first slice of an inner dimension of which `left` entries remain,
    __device__ __forceinline__ void start(const uint16_t* at, int left) {
      p = reinterpret_cast<const char*>(at);
      if (!KS) records = ((rows - 1) * ld + last) * 2;
      edge(left);
    }
    // and the one after it.
    __device__ __forceinline__ void next(int left) {
      p += KS ? (long)ld * (BK16 * 2) : (long)(BK16 * 2);
      if (!KS) records -= BK16 * 2;
      edge(left);
    }
    __device__ __forceinline__ void edge(int left) {
      if (KS) {  // rows k past the inner dimension lie past the end
        records = left > 0 ? ((min(left, BK16) - 1) * ld + last) * 2 : 0;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) base[e] = kin[e] < left ? off[e] : (int)0x80000000;
      }
    }
    // Past the last slice every load brings zeros.
    __device__ __forceinline__ void stop() { records = 0; }

    __device__ __forceinline__ void load1(int li, char* lds) const {
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, records, 0x00020000);
      const int blk = wave * LOADS + li;
      int voff;
      if (KS) {
        constexpr int CPR = ROWS / 8;         // 16-byte chunks per row
        constexpr int KPL = 64 / CPR;         // rows k per wave load
        const int k = blk * KPL + lane / CPR;
        const int c = (lane % CPR) ^ (kswz<ROWS>(k) << 1);
        voff = (k * ld + c * 8) * 2;
      } else {
        voff = base[blk & 1] + blk * 16 * ld;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(lds + blk * 1024), 16,
                                               voff, 0, 0, 0);
    }
  };

  // Four entries of a column (see above).  The restrict-qualified argument
  // gives the read an alias scope; without one the compiler takes it to
  // depend on every load into LDS in flight and waits for them all before it.
  // What it does depend on is waited for at slice_barrier.
  static __device__ __forceinline__ v4s read_tr(const char* __restrict__ p) {
    typedef __attribute__((address_space(3))) v4s* lds4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
  }

  // 16 rows x 32 k of an operand: lane l gets row l mod 16, k = 8 (l / 16) .. + 7
  template <int ROWS, bool KS>
  static __device__ __forceinline__ v8s fragment(const char* lds, int lane, int row0, int ks) {
    if (!KS) {
      const int row = row0 + (lane & 15);
      const int c = (ks * 4 + (lane >> 4)) ^ swz(row);
      return *reinterpret_cast<const v8s*>(lds + row * 128 + c * 16);
    } else {
      const int k = ks * 32 + 8 * (lane >> 4) + ((lane & 15) >> 2);
      const char* p = lds + k * (ROWS * 2) + (((row0 >> 4) ^ kswz<ROWS>(k)) << 5) + (lane & 3) * 8;
      const v4s a = read_tr(p), b = read_tr(p + 4 * ROWS * 2);
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }

  // The whole product of one tile; nprod is 1, or 3 for operands in two slices.
  //
  // Order of a slice t (two steps of 32 k): the MFMAs of a step run in fixed
  // slots, and after each slot go the LDS reads of the next step's fragments
  // (an A fragment right after its last use) and, in the second step, the
  // loads of slice t + 2.  One barrier per slice, a quarter into the second
  // step, whose MFMAs cover the latency of the last reads of buffer t mod 2;
  // this wave's loads of slice t + 1, issued a whole slice earlier, have
  // landed by then.  Reads of buffer t + 1 and loads into buffer t follow it.
  static constexpr int BAR = FM * FN / 4 - 1;
  // slot r of FM FN pressed into those after the barrier
  static constexpr int after_barrier(int r) { return BAR + 1 + r * (FM * FN - BAR - 1) / (FM * FN); }

  static __device__ __forceinline__ void run(v4f (&acc)[FM][FN], char* smem, const Source16& A, const Source16& B,
                                             int q, int nprod) {
    constexpr int SLOTS = FM * FN, LPW = A_LOADS + B_LOADS;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    Loader<BM, AKS, A_LOADS> la;
    Loader<BN, BKS, B_LOADS> lb;
    la.init(A, lane, wave);
    lb.init(B, lane, wave);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    const int nk = (q + BK16 - 1) / BK16;
    const int total = nk * nprod;
    if (total == 0) return;
    // The slices in the order they are loaded: `left` entries of the inner
    // dimension remain of product u.
    int u = 0, left = q;
    auto planes = [&]() {
      la.start(A.base + (nprod == 3 && u == 0 ? A.plane : 0), q);
      lb.start(B.base + (nprod == 3 && u == 1 ? B.plane : 0), q);
    };
    auto advance = [&]() {
      left -= BK16;
      la.next(left);
      lb.next(left);
      if (left <= 0) {
        if (++u < nprod) {
          left = q;
          planes();
        } else {
          la.stop();
          lb.stop();
        }
      }
    };
    planes();
    auto load1 = [&](int buf, int li) {
      char* d = smem + buf * BUF;
      if (li < A_LOADS)
        la.load1(li, d);
      else
        lb.load1(li - A_LOADS, d + A_BYTES);
    };
    // fragment f of step ks in buffer buf: f < FN are B's, the rest A's
    auto read1 = [&](int buf, int ks, int f) -> v8s {
      const char* As = smem + buf * BUF;
      if (f < FN) return fragment<BN, BKS>(As + A_BYTES, lane, wn * (BN / WN) + f * 16, ks);
      return fragment<BM, AKS>(As, lane, wm * (BM / WM) + (f - FN) * 16, ks);
    };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int li = 0; li < LPW; ++li) load1(b, li);
      advance();
    }
    wait_loads<LPW>();  // slice 0 (loads return in order)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    v8s cur[FM + FN], nxt[FM + FN];
#pragma unroll
    for (int f = 0; f < FM + FN; ++f) cur[f] = read1(0, 0, f);
    __builtin_amdgcn_s_waitcnt(0xc07f);

    for (int t = 0; t < total; ++t) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int rbuf = ks ? (t + 1) & 1 : t & 1;  // (past the end: zeros, not used)
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
          const int i = r / FN, j = r % FN;
          acc[i][j] = T::mfma(cur[FN + i], cur[j], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (ks && r == BAR) {
            slice_barrier();
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int f = 0; f < FM + FN; ++f) {
            const int slot = f < FN ? f * (SLOTS / FN) + 1 : (f - FN) * FN + FN - 1;
            if ((ks ? after_barrier(slot) : slot) == r) nxt[f] = read1(rbuf, 1 - ks, f);
          }
          if (ks) {
#pragma unroll
            for (int li = 0; li < LPW; ++li)
              if (after_barrier(li * SLOTS / LPW + (SLOTS > LPW)) == r) load1(t & 1, li);
            if (r == SLOTS - 1) advance();
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (ks) __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
        for (int f = 0; f < FM + FN; ++f) cur[f] = nxt[f];
      }
    }
  }
};

}  // namespace oz
