// One output tile of a product of 16-bit operands on gfx950 matrix cores:
//   acc[i][j] = sum over k of A[i][k] B[j][k]
// with the accumulators in FP32.  Shared by the grouped products
// (gemm16.hip) and the Newton-Schulz steps (ortho.hip).
//
// An operand lies "K-contiguous" (row i at i ld, its entries next to each
// other) or "K-strided" (entry (i, k) at k ld + i).  K slices of 64 entries
// go from HBM straight into LDS (16 bytes per lane) through NB buffers, in
// the operand's own order; a K-strided tile is transposed on its way from
// LDS into registers (ds_read_b64_tr_b16: 16 lanes read 4 x 16 entries and
// each receives a column of 4).  The loads carry a range check: what lies
// past the operand's end arrives as zero, and entries past the inner
// dimension of a K-contiguous row are sent past the end, so ragged edges
// cost no branch and never meet their neighbours' values.
//
// An operand may come as two slices (hi + lo, see slices.hip).  A K slice then
// holds both of both operands, and every step forms the three products lo hi,
// hi lo, hi hi into the same accumulators: three MFMAs per pair of tiles for
// four tiles loaded, where walking the products one after the other loads six.
//
// What bounds it: a 256 x 256 tile with every unit busy takes 1.4 us per slice
// of 64 (1.5 PFLOPS at the clock the power limit leaves, which falls from 2.3
// to 1.75 GHz as the matrix cores fill), 9 us besides to start and to store;
// one of 128 x 128 takes 0.6 us per slice, as two products more loads per
// operation.  Reads of LDS have no bank conflicts to speak of (0.0 to 0.2% of
// their cycles).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oz {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// Runs of a caller's array that begin at any of its entries: the hardware reads
// and writes them as one all the same (22720 rows of 1811 results in bf16: 79 us
// entry by entry where they lie on no 16-byte boundary, 42 so; in f32 158 / 95).
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef v4u v4u_any __attribute__((aligned(4)));
typedef v4f v4f_any __attribute__((aligned(4)));
typedef v4s v4s_any __attribute__((aligned(2)));
typedef v8s v8s_any __attribute__((aligned(2)));

// The sum over the parts, in their order, of four partial sums next to each
// other (zeros past `left`), the parts `apart` entries apart; eight loads in flight
// (32 parts of 64 x 64: 2 us less than one after the other).
__device__ __forceinline__ v4f sum_parts(const float* from, long apart, int parts, int left) {
  v4f v = {0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < parts; p0 += 8) {
    v4f x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float* at = from + min(p0 + u, parts - 1) * apart;
      if (left >= 4) {
        x[u] = *reinterpret_cast<const v4f_any*>(at);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[u][k] = k < left ? at[k] : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (p0 + u < parts) v += x[u];
  }
  return v;
}

struct Half {
  static constexpr int LANE = 8;  // k per lane of an operand
  typedef uint16_t Entry;
  static __device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};
struct Bfloat {
  static constexpr int LANE = 8;
  typedef uint16_t Entry;
  static __device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                   0);
  }
};

// Single precision as it is: lane l of an operand holds k = 4 (l / 16) .. + 3,
// one of which goes into each of four products (both operands alike, so the
// sum is over the same k whatever their order).
struct Single {
  static constexpr int LANE = 4;
  typedef float Entry;
  static __device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
    for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[t], y[t], c, 0, 0, 0);
    return c;
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

// This wave's LDS reads are done and all but its last AHEAD loads into LDS
// have landed; then every wave's.
template <int AHEAD>
__device__ __forceinline__ void slice_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  wait_loads<AHEAD>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Block b of `total` tiles, each XCD (b mod 8) taking a contiguous eighth.
__device__ __forceinline__ int xcd_order(int b, int total) {
  const int x = b & 7, per = total >> 3, rest = total & 7;
  return x * per + min(x, rest) + (b >> 3);
}

// Inside its run an XCD walks `major` panels GROUP at a time against all of
// `minor`, so the blocks running together share both operands' panels in L2.
template <int GROUP>
__device__ __forceinline__ void panel_order(int w, int major, int minor, int& a, int& b) {
  const int first = w / (GROUP * minor) * GROUP;
  const int in = w % (GROUP * minor);
  const int g = min(GROUP, major - first);
  a = first + in % g;
  b = in / g;
}

// Tiles (a, b), b <= a < size, of a symmetric result: GROUP rows of tiles at a
// time, down each column of them, so that blocks running together share
// panels as above (3 to 5% faster at 4096 rows than row after row of tiles).
template <int GROUP>
__device__ __forceinline__ void triangle_order(int w, int size, int& a, int& b) {
  // GROUP i rows' worth of triangle come before row group i
  int i = 0, rows = min(GROUP, size);
  while (true) {
    const int tiles = rows * GROUP * i + rows * (rows + 1) / 2;
    if (w < tiles) break;
    w -= tiles;
    ++i;
    rows = min(GROUP, size - GROUP * i);
  }
  const int first = GROUP * i;
  if (w < rows * first) {
    a = first + w % rows;
    b = w / rows;
    return;
  }
  w -= rows * first;
  int c = 0;
  while (w >= rows - c) {
    w -= rows - c;
    ++c;
  }
  a = first + c + w;
  b = first + c;
}

template <class T, int BM, int BN, int WM, int WN, bool AKS, bool BKS, int NB = 2, bool PAIR = false>
struct Tile16 {
  static constexpr int NW = WM * WN, ROWS_M = BM, ROWS_N = BN;
  static constexpr int THREADS = NW * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int PLANES = PAIR ? 2 : 1;
  static constexpr int A_BYTES = BM * BK16 * 2, B_BYTES = BN * BK16 * 2;  // of one slice of the operand
  static constexpr int BUF = PLANES * (A_BYTES + B_BYTES);
  static constexpr int SMEM = NB * BUF;
  static constexpr int A_LOADS = A_BYTES / 1024 / NW, B_LOADS = B_BYTES / 1024 / NW;
  static_assert(A_LOADS * NW * 1024 == A_BYTES && B_LOADS * NW * 1024 == B_BYTES, "whole wave loads");
  static_assert(FM * WM * 16 == BM && FN * WN * 16 == BN, "whole matrix-core tiles");

  // Which part of the tile a wavefront computes.  Wavefronts w and w + 4 share a
  // SIMD; the columns' halves are dealt so that each SIMD has both, and a tile
  // of which only the first half exists takes half the time (see resume).
  static constexpr int HALF = WN > 1 ? WN / 2 : 1;
  static __device__ __forceinline__ int wave_m(int wave) { return wave / HALF % WM; }
  static __device__ __forceinline__ int wave_n(int wave) { return wave % HALF + wave / (HALF * WM) * HALF; }

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
    int records;     // the bytes that may be read from there,
    long plane;      // the bytes from there to the low slice
    int ld;
    int off[2];      // lane's byte offset in an even and an odd load (K-contiguous)
    int kin[2];      // lane's first k within the slice
    int base[2];     // off, or past the end for a lane whose k lies past the inner dimension
    int last, rows;
    int lane, wave;

    __device__ __forceinline__ void init(const Source16& s, int lane_, int wave_) {
      ld = s.ld;
      plane = s.plane * 2;
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

    __device__ __forceinline__ void load1(int li, int low, char* lds) const {
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p + low * plane), 0, records, 0x00020000);
      const int blk = wave * LOADS + li;
      int voff;
      if (KS) {
        constexpr int CPR = ROWS / 8;         // 16-byte chunks per row
        constexpr int KPL = 64 / CPR;         // rows k per wave load
        const int k = blk * KPL + lane / CPR;
        const int c = (lane % CPR) ^ (kswz<ROWS>(k) << 1);
        voff = (k * ld + c * 8) * 2;
      } else {
        voff = ((blk & 1) ? base[1] : base[0]) + blk * 16 * ld;
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

  // MFMA slots of a step.  Long steps: per A fragment i its products with every
  // B fragment, the pair's three kinds one after the other, smallest first.
  // Short ones: all of one kind before the next, which keeps MFMAs into the
  // same accumulator apart.
  static constexpr int KINDS = PAIR ? 3 : 1;
  static constexpr int SLOTS = KINDS * FM * FN;
  static constexpr bool SHORT = SLOTS <= 24;
  static constexpr int NF = PLANES * (FM + FN);  // fragments of a step: B's (high, low), then A's (high, low of each i)
  static constexpr int LPW = PLANES * (A_LOADS + B_LOADS);

  // The slot after which fragment f of the next step is read.  Short steps
  // read them all in their first half, whose latency the second half covers;
  // in the long steps of a 256 x 256 tile each A fragment is read right after
  // its last use, so that old and new can share registers.
  static constexpr int read_slot(int f) {
    if (SHORT) return f * SLOTS / (2 * NF);
    if (f < PLANES * FN) return f * (SLOTS / (PLANES * FN)) + (SLOTS / (PLANES * FN) > 1);
    const int i = (f - PLANES * FN) / PLANES, low = (f - PLANES * FN) % PLANES;
    return (i * KINDS + (low ? 1 : KINDS)) * FN - 1;
  }
  static constexpr int load_slot(int li) { return li * SLOTS / LPW + (SLOTS > LPW); }

  // The whole product of one tile.
  //
  // Order of a slice t (two steps of 32 k): the MFMAs of a step run in fixed
  // slots, and after each slot go the LDS reads of the next step's fragments
  // and, in the second step, the loads of slice t + NB into the buffer of
  // slice t.  One barrier per slice, a quarter into the second step, whose
  // MFMAs cover the latency of the last reads of slice t; this wave's loads of
  // slice t + 1, issued NB - 1 slices earlier, have landed by then (loads
  // return in order; those of NB - 2 slices stay in flight).  Reads of slice
  // t + 1 and the loads follow it.  Two buffers are enough where a slice takes
  // longer than a load (256 x 256 tiles, or two 128 x 128 blocks on a compute
  // unit); a lone small tile's slice is over long before, and it keeps more
  // slices in flight.
  static constexpr int BAR = SLOTS >= 8 ? SLOTS / 4 - 1 : 0;
  static_assert(SLOTS >= 2, "the loads and reads of the second step follow its barrier");
  // slot r pressed into those after the barrier
  static constexpr int after_barrier(int r) { return BAR + 1 + r * (SLOTS - BAR - 1) / SLOTS; }

  // The loads of one tile's slices, in order.
  struct Feed {
    Loader<BM, AKS, A_LOADS> la;
    Loader<BN, BKS, B_LOADS> lb;
    int left;  // entries of the inner dimension from the slice to load on
    char* smem;

    __device__ __forceinline__ Feed(char* lds) : smem(lds) {}

    __device__ __forceinline__ void begin(const Source16& A, const Source16& B, int q) {
      const int lane = threadIdx.x & 63;
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      la.init(A, lane, wave);
      lb.init(B, lane, wave);
      left = q;
      la.start(A.base, left);
      lb.start(B.base, left);
      end();
    }
    __device__ __forceinline__ void end() {
      if (left <= 0) {
        la.stop();
        lb.stop();
      }
    }
    __device__ __forceinline__ void advance() {
      left -= BK16;
      la.next(left);
      lb.next(left);
      end();
    }
    // load li of a slice; a buffer holds A's high (and low) tile, then B's
    __device__ __forceinline__ void load1(int buf, int li) const {
      char* d = smem + buf * BUF;
      if (li < PLANES * A_LOADS)
        la.load1(li % A_LOADS, li / A_LOADS, d + li / A_LOADS * A_BYTES);
      else
        lb.load1((li - PLANES * A_LOADS) % B_LOADS, (li - PLANES * A_LOADS) / B_LOADS,
                 d + PLANES * A_BYTES + (li - PLANES * A_LOADS) / B_LOADS * B_BYTES);
    }
    __device__ __forceinline__ void issue(int buf) {
#pragma unroll
      for (int li = 0; li < LPW; ++li) load1(buf, li);
      advance();
    }
  };

  static __device__ __forceinline__ void run(v4f (&acc)[FM][FN], char* smem, const Source16& A, const Source16& B,
                                             int q) {
    Feed feed(smem);
    feed.begin(A, B, q);
    feed.issue(0);
    resume(acc, feed, q, BN);
  }

  // The product of the tile whose slice 0 has been issued.  SOME or twice SOME
  // more memory operations have followed it where `later` is 1 or 2; it may be
  // 0 always.  A wavefront whose columns all lie past the first `cols` only
  // loads.
  template <int SOME = 0>
  static __device__ __forceinline__ void resume(v4f (&acc)[FM][FN], Feed& feed, int q, int cols, int later = 0) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave_m(wave), wn = wave_n(wave);
    const char* smem = feed.smem;
    const int total = (q + BK16 - 1) / BK16;
    auto read1 = [&](int buf, int ks, int f) -> v8s {
      const char* As = smem + buf * BUF;
      if (f < PLANES * FN)
        return fragment<BN, BKS>(As + PLANES * A_BYTES + f / FN * B_BYTES, lane, wn * (BN / WN) + f % FN * 16, ks);
      const int i = (f - PLANES * FN) / PLANES, low = (f - PLANES * FN) % PLANES;
      return fragment<BM, AKS>(As + low * A_BYTES, lane, wm * (BM / WM) + i * 16, ks);
    };
#pragma unroll
    for (int b = 1; b < NB; ++b) feed.issue(b);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // slice 0 (loads and stores leave the counter in order)
    if (SOME > 0 && later == 2)
      wait_loads<(NB - 1) * LPW + 2 * SOME>();
    else if (SOME > 0 && later == 1)
      wait_loads<(NB - 1) * LPW + SOME>();
    else
      wait_loads<(NB - 1) * LPW>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (wn * (BN / WN) >= cols) {
      int buf = 0;
      for (int t = 0; t < total; ++t) {
        slice_barrier<(NB - 2) * LPW>();
        feed.issue(buf);
        buf = buf + 1 == NB ? 0 : buf + 1;
      }
      return;
    }
    v8s cur[NF], nxt[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) cur[f] = read1(0, 0, f);
    __builtin_amdgcn_s_waitcnt(0xc07f);

    int buf = 0;
    for (int t = 0; t < total; ++t) {
      const int following = buf + 1 == NB ? 0 : buf + 1;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int rbuf = ks ? following : buf;  // (past the end: zeros, not used)
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
          const int i = SHORT ? r / FN % FM : r / (KINDS * FN), kind = SHORT ? r / (FM * FN) : r / FN % KINDS, j = r % FN;
          const int fa = PLANES * FN + i * PLANES + (PAIR && kind == 0), fb = j + (PAIR && kind == 1 ? FN : 0);
          acc[i][j] = T::mfma(cur[fa], cur[fb], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (ks && r == BAR) {
            slice_barrier<(NB - 2) * LPW>();
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int f = 0; f < NF; ++f)
            if ((ks ? after_barrier(read_slot(f)) : read_slot(f)) == r) nxt[f] = read1(rbuf, 1 - ks, f);
          if (ks) {
#pragma unroll
            for (int li = 0; li < LPW; ++li)
              if (after_barrier(load_slot(li)) == r) feed.load1(buf, li);
            if (r == SLOTS - 1) feed.advance();
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (ks) __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
        for (int f = 0; f < NF; ++f) cur[f] = nxt[f];
      }
      buf = following;
    }
  }
};

}  // namespace oz
