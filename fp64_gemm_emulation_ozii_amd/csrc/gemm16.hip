// Products over ragged groups in 16-bit slices (tile16.h).
//
//   grouped:  C(:, j) = op(A_e) B(:, j)          for j in J_e
//   outer:    C_e = sum over j in J_e of A(:, j) B(:, j)^T
//
// J_e are the groups of groups.h, known on the device only: a launch has a
// fixed number of blocks for the compute units, which share out the tiles that
// the offsets make (share.h), and a block looks a tile up in them (one
// wavefront-wide scan per 64 groups).  Groups of few columns have kernels of
// their own, which stream the weights (few_columns_kernel).
#include <algorithm>
#include <cmath>

#include "groups.h"
#include "products.h"
#include "share.h"
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

// Four consecutive rows of a column of C.
__device__ __forceinline__ void store4(const Grouped16& g, long col, int row, v4f v) {
  const long to = col * g.ldc + row;
  if (g.ctype == OZGEMM_F32) {
    float* out = (float*)g.C + to;
    if (row + 4 <= g.m) {
      *reinterpret_cast<v4f_any*>(out) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row + k < g.m) out[k] = v[k];
    }
  } else {
    v4s h;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = (short)round16(v[k], g.ctype);
    short* out = (short*)g.C + to;
    if (row + 4 <= g.m) {
      *reinterpret_cast<v4s_any*>(out) = h;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row + k < g.m) out[k] = h[k];
    }
  }
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

// A tile to compute: its operands, its inner dimension and where it goes.
struct Job {
  Source16 A, B;
  int inner;
  Target to;
};

// A block's tiles.  The next tile's first slice lands in buffer 0 while this
// one's results go out through the LDS behind it, and its products begin
// before they are written (16384 rows, 32 groups of 4096 x 2048: 357 us with a
// block per tile, 326 so, call after call; 330 to 430 in single calls).  place(L, dm, dn) gives the job of tile L from
// (dm, dn) in it on.
template <class Tile, class Small>
struct Walk {
  using Out = Store<Tile>;
  static constexpr int STAGE = Tile::BUF;
  static constexpr int SMEM = STAGE + (Tile::BUF > Out::BYTES ? Tile::BUF : Out::BYTES);
  static_assert(Small::SMEM <= SMEM && Store<Small>::BYTES <= SMEM, "quarter tiles use the same LDS");

  template <class Place>
  static __device__ __forceinline__ void run(char* smem, int total, int units, int skip, Place place) {
    constexpr int BT = Tile::ROWS_M;
    static_assert(BT == Tile::ROWS_N && BT == 2 * Small::ROWS_M && BT == 2 * Small::ROWS_N, "square tiles and quarters");
    const Share share = share_of(total, units, blockIdx.x + skip);
    if (share.first < 0) return;
    if (share.quarter >= 0) {
      const Job job = place(share.first, (share.quarter & 1) * (BT / 2), (share.quarter >> 1) * (BT / 2));
      if (job.to.m0 >= job.to.m || job.to.n0 >= job.to.n_end) return;
      v4f acc[Small::FM][Small::FN];
      Small::run(acc, smem, job.A, job.B, job.inner);
      slice_barrier<0>();
      Store<Small>::run(acc, smem, job.to);
      return;
    }
    typename Tile::Feed feed(smem);
    Job job = place(share.first, 0, 0);
    feed.begin(job.A, job.B, job.inner);
    feed.issue(0);
    v4f acc[Tile::FM][Tile::FN];
    int later = 0;
    for (int round = 1, L = share.first;; ++round) {
      Tile::template resume<Out::STORES>(acc, feed, job.inner, job.to.n_end - job.to.n0, later);
      const Target from = job.to;
      slice_barrier<0>();  // every wave has read its last operands, and no load into LDS is in flight
      const bool more = round < share.rounds;
      if (more) {
        L += units;
        job = place(L, 0, 0);
        feed.begin(job.A, job.B, job.inner);
        feed.issue(0);
      }
      Out::run(acc, smem + STAGE, from);
      if (!more) break;
      later = Out::stores(from, BT, BT);
      __builtin_amdgcn_s_barrier();  // every wave has read its staged results
      asm volatile("" ::: "memory");
    }
  }
};

// Bound by the matrix cores and, long, by the power they draw: 32768 bf16 rows,
// 16 groups of 4096 x 2048 take 555 us (990 TFLOPS, 53% of the MFMA cycles at
// the 1.75 GHz the power leaves; 59% where the weights lie K-strided).  A tile
// is 256 rows of the weights by 256 columns of one group, of which the last of
// a group is half empty on average: 512 rows a group run at 840 TFLOPS.  Tiles
// are walked group by group, four panels of columns against all rows of the
// weights at a time on an XCD, so that weights come from HBM about once (536 MB
// read for 537 MB of weights and 67 MB of rows, most of which stay in L2).
// F32 (PAIR) holds two slices of both operands and takes 128 x 128: 8192 rows,
// 16 groups of 2048 x 2048 take 295 us, 233 TFLOPS of f32 or 700 of its slices.
template <class T, int BT, bool AKS, bool PAIR>
__global__ __launch_bounds__(512) void grouped_n_kernel(Grouped16 g) {
  using Tiles = Walk<Tile16<T, BT, BT, 2, 4, AKS, false, 2, PAIR>, Tile16<T, BT / 2, BT / 2, 2, 4, AKS, false, 4, PAIR>>;
  __shared__ __attribute__((aligned(1024))) char smem[Tiles::SMEM];
  const int tiles_m = (g.m + BT - 1) / BT;
  const GroupIndex index(g.offsets, g.groups, g.n, BT);
  const int whole = tiles_m * index.total, total = whole * g.parts;
  // a part's inner dimension: whole slices
  const int each = ((g.q + BK16 - 1) / BK16 + g.parts - 1) / g.parts * BK16;
  Tiles::run(smem, total, g.units, g.skip, [&](int L, int dm, int dn) {
    const int part = L / whole, k0 = min(part * each, g.q);
    int nj, mi;
    panel_order<4>(xcd_order(L - part * whole, whole), index.total, tiles_m, nj, mi);
    const GroupTile gt = index.find(nj);
    const int m0 = mi * BT + dm, n0 = gt.begin + dn;
    const long a_at = AKS ? k0 * g.A.ld + m0 : m0 * g.A.ld + k0;
    return Job{Source16{g.A.p + gt.group * g.A.batch + a_at, g.A.plane, (int)g.A.ld, g.m - m0,
                        (int)g.A.last - (AKS ? m0 : k0)},
               Source16{g.B.p + n0 * g.B.ld + k0, g.B.plane, (int)g.B.ld, gt.end - n0, (int)g.B.last - k0},
               min(each, g.q - k0),
               g.parts > 1 ? Target{g.partial + (long)part * g.n * g.m, OZGEMM_F32, g.m, m0, g.m, n0, gt.end, nullptr,
                                    nullptr}
                           : Target{g.C, g.ctype, g.ldc, m0, g.m, n0, gt.end,
                                    g.A.ex ? g.A.ex + gt.group * g.A.ex_batch : nullptr, g.B.ex}};
  });
}

// The sum of the parts, in their order, into the columns of the groups: a
// block per 64 columns of a group and 64 rows.
__global__ __launch_bounds__(256) void join_columns_kernel(Grouped16 g) {
  const GroupIndex index(g.offsets, g.groups, g.n, 64);
  if ((int)blockIdx.x >= index.total) return;
  const GroupTile gt = index.find(blockIdx.x);
  const int row = blockIdx.y * 64 + (threadIdx.x & 15) * 4;
  if (row >= g.m) return;
  const int32_t* ea = g.A.ex ? g.A.ex + gt.group * g.A.ex_batch : nullptr;
  for (int col = gt.begin + (threadIdx.x >> 4); col < min(gt.end, gt.begin + 64); col += 16) {
    v4f v = sum_parts(g.partial + (long)col * g.m + row, (long)g.n * g.m, g.parts, g.m - row);
    if (ea != nullptr) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = unscale(v[k], ea[min(row + k, g.m - 1)], g.B.ex[col]);
    }
    store4(g, col, row, v);
  }
}

// Both operands K-strided in place (F32 and what is not aligned: K-contiguous
// slices, each group padded to whole slices).  Bound like grouped_n_kernel:
// 32768 bf16 rows, 16 groups of 4096 x 2048 take 576 us (955 TFLOPS).
template <class T, int BT, bool KS, bool PAIR>
__global__ __launch_bounds__(512) void grouped_k_kernel(Grouped16 g) {
  using Tiles = Walk<Tile16<T, BT, BT, 2, 4, KS, KS, 2, PAIR>, Tile16<T, BT / 2, BT / 2, 2, 4, KS, KS, 4, PAIR>>;
  __shared__ __attribute__((aligned(1024))) char smem[Tiles::SMEM];
  const int tiles_m = (g.m + BT - 1) / BT, tiles_q = (g.q + BT - 1) / BT;
  const int per = tiles_m * tiles_q, whole = per * g.groups, total = whole * g.parts;
  const GroupIndex index(g.offsets, g.groups, g.n, BK16);
  Tiles::run(smem, total, g.units, g.skip, [&](int L, int dm, int dn) {
    const int part = L / whole;
    L -= part * whole;
    // Every XCD takes an eighth of each group's tiles: the groups' lengths
    // differ, and an XCD with whole groups of its own waited for the longest.
    const int x = L & 7, i = L >> 3, eighth = per >> 3;
    const int e = per % 8 == 0 ? i / eighth : L / per;
    int mi, qj;
    panel_order<4>(per % 8 == 0 ? x * eighth + i % eighth : L % per, tiles_m, tiles_q, mi, qj);
    const GroupTile gt = index.at(e);
    const int m0 = mi * BT + dm, q0 = qj * BT + dn;
    // this part's columns: whole slices of the group's
    const int slices = (gt.end - gt.begin + BK16 - 1) / BK16, each = (slices + g.parts - 1) / g.parts;
    const int from = min(part * each, slices) * BK16, len = min(gt.end - gt.begin - from, each * BK16);
    // K-strided: the group's columns; else padded planes, where they begin at 64 x its tiles before
    const int k0 = (KS ? gt.begin : gt.first * BK16) + from;
    const long a_at = KS ? k0 * g.A.ld + m0 : m0 * g.A.ld + k0, b_at = KS ? k0 * g.B.ld + q0 : q0 * g.B.ld + k0;
    return Job{Source16{g.A.p + a_at, g.A.plane, (int)g.A.ld, g.m - m0, (int)g.A.last - (KS ? m0 : k0)},
               Source16{g.B.p + b_at, g.B.plane, (int)g.B.ld, g.q - q0, (int)g.B.last - (KS ? q0 : k0)},
               len <= 0 ? 0 : KS ? len : (len + BK16 - 1) / BK16 * BK16,
               g.parts > 1 ? Target{g.partial + ((long)part * g.groups + e) * g.m * g.q, OZGEMM_F32, g.m, m0, g.m, q0,
                                    g.q, nullptr, nullptr}
                           : Target{(char*)g.C + (size_t)e * g.cbatch * (g.ctype == OZGEMM_F32 ? 4 : 2), g.ctype,
                                    g.ldc, m0, g.m, q0, g.q, g.A.ex ? g.A.ex + e * g.A.ex_batch : nullptr,
                                    g.B.ex ? g.B.ex + e * g.B.ex_batch : nullptr}};
  });
}

// Groups of a few columns: bound by reading the weights once.  A block takes
// 16 MR rows of a group's weights and up to 64 of its columns; its eight
// wavefronts share the inner dimension, 32 DEPTH entries of it at a time,
// whose loads are all in flight before the first product, straight from HBM
// into the MFMA's operand layout (16 rows x 64 bytes per load; the two halves
// of a 128-byte line are loaded one after the other).  The columns, which the
// L2 serves, come the same way.  The wavefronts' sums meet in LDS.  256 rows
// over 32 groups of 4096 x 2048 in bf16 take 106 us, 5.0 TB/s of weights; one
// token's 8 rows over 64 groups of 1024 x 2048 take 9.3 us, 3.6 TB/s, of which
// launch, look-up and the first load's latency are half.  Single
// precision goes without slices: at so few columns its matrix-core rate is
// enough, and cutting the weights would read and write them three times over.
//
// Where the tiles of a product leave units idle and its inner dimension is
// long, blocks share that too, in parts whose sums join_columns_kernel adds.
// Rows (K-strided weights: 16 x the entries in 16 bytes) and columns of a tile:
constexpr int FEW_MR = 2, FEW_ROWS = 16 * FEW_MR, FEW_COLS = 64, FEW_KS_COLS = 32;

struct FewTile {
  bool any;       // this block has a tile
  int tile, m0;   // of the columns; first row
  int k0, k_end;  // its part of the inner dimension
};

template <int ROWS, int CHUNK>
__device__ __forceinline__ FewTile few_tile(Grouped16& g, const GroupIndex& index) {
  const int tiles_m = (g.m + ROWS - 1) / ROWS, whole = tiles_m * index.total;
  FewTile t{};
  const int part = whole > 0 ? (int)blockIdx.x / whole : g.parts;
  t.any = part < g.parts;
  const int L = whole > 0 ? (int)blockIdx.x % whole : 0;
  t.tile = L / tiles_m;
  t.m0 = L % tiles_m * ROWS;
  const int chunks = (g.q + CHUNK - 1) / CHUNK, per = (chunks + g.parts - 1) / g.parts * CHUNK;
  t.k0 = part * per;
  t.k_end = min(t.k0 + per, g.q);
  if (g.parts > 1) {  // (the sum of an empty part is stored too)
    g.C = g.partial + (long)part * g.n * g.m;
    g.ctype = OZGEMM_F32;
    g.ldc = g.m;
  }
  return t;
}

// N entries next to each other, of a row of `length` entries of which `left`
// are left; zeros follow where those are fewer.  EDGE: they may be, and may
// lie on no 16-byte boundary.  Then the row's last N entries are read and moved
// down.  AROUND: 16-bit entries come as the 32-bit words around them (1 of
// 1023 x 1023, 64 rows: 23 us with reads that begin in the middle of a word, 13
// so; where lanes read next to each other, as in few_outer_kernel, the further
// reads cost more than that: 46 us against 68 for 4096 rows).  load() issues
// the reads, get() works on what they brought, after all that are to be in flight.
template <class E, int N, bool EDGE, bool AROUND = EDGE && sizeof(E) == 2>
struct Run {
  static constexpr int WORDS = N * (int)sizeof(E) / 4;
  typedef E Entries __attribute__((ext_vector_type(N)));
  typedef uint32_t Words __attribute__((ext_vector_type(WORDS), may_alias));
  typedef Words Loose __attribute__((aligned(AROUND ? 4 : sizeof(E))));
  typedef uint32_t Word __attribute__((may_alias));
  Words w;
  uint32_t after;  // the word after them, where the entries begin in the middle of one

  __device__ __forceinline__ void load(const E* p, int left, int length) {
    w = Words{};
    after = 0;
    if (left <= 0) return;
    if (!EDGE) {
      w = *reinterpret_cast<const Words*>(p);
    } else if (length >= N) {
      p -= max(N - left, 0);
      if (AROUND) {
        const Word* from = reinterpret_cast<const Word*>((uintptr_t)p & ~(uintptr_t)3);
        w = *reinterpret_cast<const Loose*>(from);
        after = from[WORDS - 1 + (((uintptr_t)p >> 1) & 1)];
      } else {
        w = *reinterpret_cast<const Loose*>(p);
      }
    } else {
      Entries r = {};
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) r[i] = p[i];
      w = __builtin_bit_cast(Words, r);
    }
  }

  __device__ __forceinline__ Entries get(const E* p, int left, int length) const {
    Words v = w;
    if (EDGE && left > 0 && length >= N) {
      const int over = max(N - left, 0);
      if (AROUND) {
        const int half = ((uintptr_t)(p - over) & 2) * 8;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
          v[i] = __builtin_amdgcn_alignbit(i + 1 < WORDS ? v[i + 1 < WORDS ? i + 1 : i] : after, v[i], half);
      }
      if (__ballot(over > 0) != 0) {
        const int words = over * (int)sizeof(E) / 4;
        const int half = over * (int)sizeof(E) % 4 * 8;
#pragma unroll
        for (int by = 1; by < WORDS; by *= 2) {
          if (words & by) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) v[i] = i + by < WORDS ? v[i + by < WORDS ? i + by : i] : 0;
          }
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
          v[i] = __builtin_amdgcn_alignbit(i + 1 < WORDS ? v[i + 1 < WORDS ? i + 1 : i] : 0, v[i], half);
      }
    }
    return __builtin_bit_cast(Entries, v);
  }
};

template <class T, int MR, int DEPTH, bool EDGE>
__global__ __launch_bounds__(512, 2) void few_columns_kernel(Grouped16 g) {
  constexpr int ROWS = 16 * MR, COLS = FEW_COLS, CF = COLS / 16, WAVES = 8, STEP = 4 * T::LANE;
  typedef typename T::Entry Entry;
  __shared__ float sums[WAVES][16][ROWS + 4];
  const GroupIndex index(g.offsets, g.groups, g.n, COLS);
  const FewTile t = few_tile<ROWS, WAVES * STEP * DEPTH>(g, index);
  if (!t.any) return;
  const int m0 = t.m0;
  const GroupTile gt = index.find(t.tile);
  const int n0 = gt.begin, cols = min(gt.end - n0, COLS), frags = (cols + 15) / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kl = wave * STEP * DEPTH + (lane >> 4) * T::LANE;  // this lane's first k in a chunk
  // rows past the end read the last one again (their sums are not stored)
  const Entry* a[MR];
#pragma unroll
  for (int i = 0; i < MR; ++i)
    a[i] = (const Entry*)g.A.p + gt.group * g.A.batch + (long)min(m0 + i * 16 + (lane & 15), g.m - 1) * g.A.ld + kl;
  const Entry* b[CF];
#pragma unroll
  for (int c = 0; c < CF; ++c) b[c] = (const Entry*)g.B.p + (long)(n0 + min(c * 16 + (lane & 15), cols - 1)) * g.B.ld + kl;
  v4f acc[MR][CF] = {};
  for (int k0 = t.k0; k0 < t.k_end; k0 += WAVES * STEP * DEPTH) {
    const int left = g.q - kl - k0;  // entries from this lane's first on
    Run<Entry, T::LANE, EDGE> av[DEPTH][MR];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int i = 0; i < MR; ++i)
        av[d][i].load(a[i] + k0 + d * STEP, left - d * STEP, g.q);
#pragma unroll
    for (int c = 0; c < CF; ++c) {
      if (c >= frags) break;
      Run<Entry, T::LANE, EDGE> bv[DEPTH];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) bv[d].load(b[c] + k0 + d * STEP, left - d * STEP, g.q);
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const v8s fb = __builtin_bit_cast(v8s, bv[d].get(b[c] + k0 + d * STEP, left - d * STEP, g.q));
#pragma unroll
        for (int i = 0; i < MR; ++i)
          acc[i][c] = T::mfma(__builtin_bit_cast(v8s, av[d][i].get(a[i] + k0 + d * STEP, left - d * STEP, g.q)), fb,
                              acc[i][c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CF; ++c) {
    if (c >= frags) break;
#pragma unroll
    for (int i = 0; i < MR; ++i)
      *reinterpret_cast<v4f*>(&sums[wave][lane & 15][i * 16 + 4 * (lane >> 4)]) = acc[i][c];
    __syncthreads();
    const int r = threadIdx.x % (ROWS / 4) * 4, col = threadIdx.x / (ROWS / 4);
    if (col < 16 && c * 16 + col < cols && m0 + r < g.m) {
      v4f v = *reinterpret_cast<const v4f*>(&sums[0][col][r]);
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const v4f*>(&sums[w][col][r]);
      store4(g, n0 + c * 16 + col, m0 + r, v);
    }
    __syncthreads();
  }
}

// The same for weights that lie K-strided (m entries next to each other).  A
// wavefront takes 16 V rows, V the entries of 16 bytes: a lane reads V of them
// of one k (16 lanes: 256 bytes next to each other), of V k in turn, and
// transposes its V x V entries in registers into V MFMA operands, the u-th of
// which has rows m0 + V i + u, i = 0..15.  Eight wavefronts share the inner
// dimension.
template <class T, int DEPTH, bool EDGE>
__global__ __launch_bounds__(512, 2) void few_columns_ks_kernel(Grouped16 g) {
  constexpr int V = T::LANE, ROWS = 16 * V, COLS = FEW_KS_COLS, CF = COLS / 16, WAVES = 8, STEP = 4 * V;
  typedef typename T::Entry Entry;
  typedef Run<Entry, V, EDGE> Piece;
  __shared__ float sums[WAVES][16][ROWS + 4];
  const GroupIndex index(g.offsets, g.groups, g.n, COLS);
  const FewTile t = few_tile<ROWS, WAVES * STEP * DEPTH>(g, index);
  if (!t.any) return;
  const int m0 = t.m0;
  const GroupTile gt = index.find(t.tile);
  const int n0 = gt.begin, cols = min(gt.end - n0, COLS), frags = (cols + 15) / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kl = wave * STEP * DEPTH + (lane >> 4) * V;  // this lane's first k in a chunk
  const long ld = g.A.ld;
  // rows past the end read the last V again (EDGE: nothing); their sums are not stored
  const int row = m0 + (lane & 15) * V, rows = EDGE ? g.m - row : V;
  const Entry* a = (const Entry*)g.A.p + gt.group * g.A.batch + (EDGE ? row : min(row, g.m - V));
  const Entry* b[CF];
#pragma unroll
  for (int c = 0; c < CF; ++c) b[c] = (const Entry*)g.B.p + (long)(n0 + min(c * 16 + (lane & 15), cols - 1)) * g.B.ld + kl;
  v4f acc[CF][V] = {};
  for (int k0 = t.k0; k0 < t.k_end; k0 += WAVES * STEP * DEPTH) {
    Piece av[DEPTH][V], bv[DEPTH][CF];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int k = kl + k0 + d * STEP;
#pragma unroll
      for (int i = 0; i < V; ++i) av[d][i].load(a + (k + i) * ld, k + i < g.q ? rows : 0, g.m);
#pragma unroll
      for (int c = 0; c < CF; ++c) bv[d][c].load(b[c] + k0 + d * STEP, c < frags ? g.q - k : 0, g.q);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int k = kl + k0 + d * STEP;
      typename Piece::Entries at[V];
#pragma unroll
      for (int i = 0; i < V; ++i) at[i] = av[d][i].get(a + (k + i) * ld, k + i < g.q ? rows : 0, g.m);
      v8s fb[CF];
#pragma unroll
      for (int c = 0; c < CF; ++c)
        fb[c] = __builtin_bit_cast(v8s, bv[d][c].get(b[c] + k0 + d * STEP, c < frags ? g.q - k : 0, g.q));
#pragma unroll
      for (int u = 0; u < V; ++u) {
        typename Piece::Entries f;
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = at[i][u];
#pragma unroll
        for (int c = 0; c < CF; ++c) acc[c][u] = T::mfma(__builtin_bit_cast(v8s, f), fb[c], acc[c][u]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CF; ++c) {
    if (c >= frags) break;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < V; u += 4)
        *reinterpret_cast<v4f*>(&sums[wave][lane & 15][(4 * (lane >> 4) + r) * V + u]) =
            v4f{acc[c][u][r], acc[c][u + 1][r], acc[c][u + 2][r], acc[c][u + 3][r]};
    __syncthreads();
    const int r = threadIdx.x % (ROWS / 4) * 4, col = threadIdx.x / (ROWS / 4);
    if (col < 16 && c * 16 + col < cols && m0 + r < g.m) {
      v4f v = *reinterpret_cast<const v4f*>(&sums[0][col][r]);
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const v4f*>(&sums[w][col][r]);
      store4(g, n0 + c * 16 + col, m0 + r, v);
    }
    __syncthreads();
  }
}

hipError_t join_columns(const Grouped16& g, hipStream_t st) {
  hipLaunchKernelGGL(join_columns_kernel, dim3((unsigned)group_tiles_max(g.n, g.groups, 64), (unsigned)((g.m + 63) / 64)),
                     dim3(256), 0, st, g);
  return hipGetLastError();
}

long few_blocks(bool ks, int lane, int groups, int m, int n) {
  const long rows = ks ? 16 * lane : FEW_ROWS;
  return group_tiles_max(n, groups, ks ? FEW_KS_COLS : FEW_COLS) * ((m + rows - 1) / rows);
}

// 32 experts of 4096 x 2048 (16-bit), 8 / 32 rows each: MR 2, DEPTH 4 takes 111 / 147 us,
// 4, 4: 125 / 148; 1, 8: 134 / 206; 2, 8 (fewer blocks on a unit): 146 / 197.
// K-strided f32, 1 of 1024 x 2048, 128 rows: DEPTH 2 takes 26 us, 4: 30.
template <class T, bool EDGE>
hipError_t few_columns(const Grouped16& g, hipStream_t st) {
  const unsigned blocks = (unsigned)(few_blocks(g.A.ks, T::LANE, g.groups, g.m, g.n) * g.parts);
  if (g.A.ks)
    hipLaunchKernelGGL((few_columns_ks_kernel<T, 2, EDGE>), dim3(blocks), dim3(512), 0, st, g);
  else
    hipLaunchKernelGGL((few_columns_kernel<T, FEW_MR, 4, EDGE>), dim3(blocks), dim3(512), 0, st, g);
  return g.parts > 1 ? join_columns(g, st) : hipGetLastError();
}

template <class T>
hipError_t few(const Grouped16& g, hipStream_t st) {
  return g.edge ? few_columns<T, true>(g, st) : few_columns<T, false>(g, st);
}

template <class T, int BT, bool AKS, bool PAIR>
hipError_t grouped_n(Grouped16 g, hipStream_t st) {
  const hipError_t err = device_units(&g.units);
  if (err != hipSuccess) return err;
  g.skip = shares_without(group_tiles_max(g.n, g.groups, BT) * ((g.m + BT - 1) / BT) * g.parts, g.units);
  hipLaunchKernelGGL((grouped_n_kernel<T, BT, AKS, PAIR>), dim3(SHARES * g.units - g.skip), dim3(512), 0, st, g);
  return g.parts > 1 ? join_columns(g, st) : hipGetLastError();
}

// Outer products too small for the tiles, or of operands that those would
// have to be copied for: 64 x 64 entries of a group's result per block, the
// eight wavefronts share the group's columns.  A lane reads runs of 4 entries
// of LANE columns of both operands and transposes them in registers into four
// MFMA operands each: the u-th has rows m0 + 4 i + u, i = 0..15.  Bound by the
// latency of its loads, which go straight from memory into registers, a chunk
// of 256 columns (f32 128) after the other: 4096 rows of 1024 x 1024 in bf16
// take 30 us (286 TFLOPS), in f32 106 (81 TFLOPS, half the matrix cores' rate).
constexpr int FEW_OUTER = 64;

template <class T, bool EDGE>
__global__ __launch_bounds__(512, 2) void few_outer_kernel(Grouped16 g) {
  constexpr int R = 4, V = T::LANE, WAVES = 8, STEP = 4 * V, CHUNK = WAVES * STEP;
  typedef typename T::Entry Entry;
  typedef Run<Entry, R, EDGE, false> Piece;
  typedef Entry Operand __attribute__((ext_vector_type(V)));
  __shared__ float sums[WAVES][16][FEW_OUTER + 4];
  const int tiles_m = (g.m + FEW_OUTER - 1) / FEW_OUTER, tiles_q = (g.q + FEW_OUTER - 1) / FEW_OUTER;
  const int per = tiles_m * tiles_q, whole = per * g.groups;
  const int part = blockIdx.x / whole, e = blockIdx.x % whole / per, tile = blockIdx.x % per;
  const int m0 = tile % tiles_m * FEW_OUTER, q0 = tile / tiles_m * FEW_OUTER;
  const GroupTile gt = group_at(g.offsets, g.groups, g.n, CHUNK, e);
  const int chunks = (gt.end - gt.begin + CHUNK - 1) / CHUNK, each = (chunks + g.parts - 1) / g.parts * CHUNK;
  const int from = gt.begin + part * each, to = min(from + each, gt.end);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // rows past the end read the last ones again (EDGE: nothing); their sums are not stored
  const int row = m0 + (lane & 15) * R, col = q0 + (lane & 15) * R;
  const int rows = EDGE ? g.m - row : R, cols = EDGE ? g.q - col : R;
  const Entry* a = (const Entry*)g.A.p + (EDGE ? row : min(row, g.m - R));
  const Entry* b = (const Entry*)g.B.p + (EDGE ? col : min(col, g.q - R));
  v4f acc[R][R] = {};
  for (int k0 = from; k0 < to; k0 += CHUNK) {
    const int k = k0 + wave * STEP + (lane >> 4) * V;
    Piece ap[V], bp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ap[i].load(a + (long)(k + i) * g.A.ld, k + i < to ? rows : 0, g.m);
      bp[i].load(b + (long)(k + i) * g.B.ld, k + i < to ? cols : 0, g.q);
    }
    typename Piece::Entries av[V], bv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      av[i] = ap[i].get(a + (long)(k + i) * g.A.ld, k + i < to ? rows : 0, g.m);
      bv[i] = bp[i].get(b + (long)(k + i) * g.B.ld, k + i < to ? cols : 0, g.q);
    }
    v8s fb[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      Operand f;
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = bv[i][u];
      fb[u] = __builtin_bit_cast(v8s, f);
    }
#pragma unroll
    for (int u = 0; u < R; ++u) {
      Operand f;
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = av[i][u];
#pragma unroll
      for (int w = 0; w < R; ++w) acc[w][u] = T::mfma(__builtin_bit_cast(v8s, f), fb[w], acc[w][u]);
    }
  }
  if (g.parts > 1) {  // (the sum of an empty part is stored too)
    g.C = g.partial + ((long)part * g.groups + e) * g.m * g.q;
    g.ctype = OZGEMM_F32;
    g.ldc = g.m;
  } else {
    g.C = (char*)g.C + (size_t)e * g.cbatch * (g.ctype == OZGEMM_F32 ? 4 : 2);
  }
  const int waves = max(min((to - from + STEP - 1) / STEP, WAVES), 1);  // the others had no columns
#pragma unroll
  for (int w = 0; w < R; ++w) {
    if (wave < waves) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<v4f*>(&sums[wave][lane & 15][(4 * (lane >> 4) + r) * R]) =
            v4f{acc[w][0][r], acc[w][1][r], acc[w][2][r], acc[w][3][r]};
    }
    __syncthreads();
    const int r = threadIdx.x % (FEW_OUTER / 4) * 4, c = threadIdx.x / (FEW_OUTER / 4);
    if (c < 16 && q0 + c * R + w < g.q && m0 + r < g.m) {
      v4f v = *reinterpret_cast<const v4f*>(&sums[0][c][r]);
#pragma unroll
      for (int x = 1; x < WAVES; ++x)
        if (x < waves) v += *reinterpret_cast<const v4f*>(&sums[x][c][r]);
      store4(g, q0 + c * R + w, m0 + r, v);
    }
    __syncthreads();
  }
}

// The sum of the parts, in their order, into C.
__global__ __launch_bounds__(256) void join_parts_kernel(Grouped16 g) {
  const int runs = (g.m + 3) / 4;
  const long at = (long)blockIdx.x * 256 + threadIdx.x;
  if (at >= (long)runs * g.q * g.groups) return;
  const int row = (int)(at % runs) * 4, col = (int)(at / runs % g.q);
  const long e = at / runs / g.q;
  v4f v = sum_parts(g.partial + (e * g.q + col) * g.m + row, (long)g.groups * g.q * g.m, g.parts, g.m - row);
  if (g.A.ex != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = unscale(v[k], g.A.ex[e * g.A.ex_batch + min(row + k, g.m - 1)], g.B.ex[e * g.B.ex_batch + col]);
  }
  g.C = (char*)g.C + (size_t)e * g.cbatch * (g.ctype == OZGEMM_F32 ? 4 : 2);
  store4(g, col, row, v);
}

hipError_t join_parts(const Grouped16& g, hipStream_t st) {
  const long threads = (long)((g.m + 3) / 4) * g.q * g.groups;
  hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, g);
  return hipGetLastError();
}

long few_outer_blocks(int groups, int m, int q) {
  return (long)((m + FEW_OUTER - 1) / FEW_OUTER) * ((q + FEW_OUTER - 1) / FEW_OUTER) * groups;
}

template <class T>
hipError_t few_outer(const Grouped16& g, hipStream_t st) {
  const unsigned blocks = (unsigned)(few_outer_blocks(g.groups, g.m, g.q) * g.parts);
  if (g.edge)
    hipLaunchKernelGGL((few_outer_kernel<T, true>), dim3(blocks), dim3(512), 0, st, g);
  else
    hipLaunchKernelGGL((few_outer_kernel<T, false>), dim3(blocks), dim3(512), 0, st, g);
  return g.parts > 1 ? join_parts(g, st) : hipGetLastError();
}

template <class T, int BT, bool KS, bool PAIR>
hipError_t grouped_k(Grouped16 g, hipStream_t st) {
  const hipError_t err = device_units(&g.units);
  if (err != hipSuccess) return err;
  g.skip = shares_without((long)((g.m + BT - 1) / BT) * ((g.q + BT - 1) / BT) * g.groups * g.parts, g.units);
  hipLaunchKernelGGL((grouped_k_kernel<T, BT, KS, PAIR>), dim3(SHARES * g.units - g.skip), dim3(512), 0, st, g);
  return g.parts > 1 ? join_parts(g, st) : hipGetLastError();
}

}  // namespace

// (256 units: the rules below also size workspaces, which a host without a GPU may
// ask for, so they are written for the card and do not ask the device.)
//
// Whether the kernels for few columns are the faster ones: 0, or the parts in
// which they take the inner dimension.  The others cut F32 and copy operands
// off the 16-byte grid (`edge`) first.  Measured in us (few columns / tiles),
// calls from the host, which takes 12:
//
// Where their blocks are no more than the units, a call takes a block's time:
// about 1 ns per entry of the inner dimension and (1 + columns / 16), twice
// that in f32, half as much again K-strided (f32: twice) or off the grid; so
// parts of 8 us are made while units are idle.  Beyond 15 us (two columns of
// MFMA tiles: 40) the 16-bit tiles are faster, unless they wait for copies.
//   16-bit   1 of 1024 x 2048, 128 rows 15 / 17;  x 8192, 32 rows 20 / 22;  x 32768, 32 rows 29 / 37,
//            256 rows 76 / 45;  1 of 1023 x 1023, 64 rows 13 / 21;  1 of 2047 x 2047, 64 rows 21 / 31
//   f32      1 of 1024 x 2048, 128 rows 26 / 32;  x 8192, 32 rows 23 / 69;  x 32768, 32 rows 47 / 216,
//            256 rows 210 / 300
// Where they are some times more, it takes that many rounds of blocks, each
// with a fixed time besides, against the tiles' launches:
//   16-bit   16 of 512 x 512, 4096 rows 20 / 12;  64 of 128 x 128, 32768 rows 27 / 15
//   copied   1 of 255 x 511, 4096 rows 23 / 23;  2 of 1399 x 89, 4096 rows 86 / 31
//   f32      8 of 256 x 256, 4096 rows 17 / 18;  64 of 128 x 128, 32768 rows 54 / 41
// Where they are many and the columns few, they read the weights at the card's
// rate and the columns once for every 32 or 128 rows; the tiles read both from
// L2 but need many in flight for that rate:
//   16-bit  32 of 4096 x 2048   8 rows each 111 / 135   24: 131 / 139   32: 147 / 141
//           64 of 1024 x 2048   8:  60 / 71             24:  72 / 73    32:  76 / 74
//            8 of 2048 x 2048   8:  17 / 33             48:  26 / 36    64:  44 / 37
//   f32     32 of 2048 x 2048   8: 127 / 345            48: 239 / 362   96: 416 / 377
//            8 of 2048 x 2048   8:  35 / 88             48:  65 / 92    64: 109 / 93
int few_columns_parts(bool f32, bool edge, bool ks, int groups, int m, int n, int q) {
  const bool copies = f32 || edge;
  const long units = 256, blocks = few_blocks(ks, f32 ? 4 : 8, groups, m, n);
  if (blocks >= 1L << 23) return 0;  // a launch has fewer than 2^32 threads
  const long frags = std::min<long>((((long)n + groups - 1) / groups + 15) / 16, (ks ? FEW_KS_COLS : FEW_COLS) / 16);
  const long ns = (long)q * (1 + frags) * (f32 ? 2 : 1);
  if (blocks <= units) {
    const double slower = (ks ? (f32 ? 2 : 1.5) : 1) * (edge ? 1.5 : 1);
    const long parts = std::max(std::min({(long)(ns * slower / 8000), units / std::max(blocks, 1L), 32L}), 1L);
    return copies || ns / parts <= (frags > 2 ? 15000 : 40000) ? (int)parts : 0;
  }
  const long fixed = ks ? (f32 ? 4500 : 6500) : f32 ? (edge ? 8500 : 5500) : edge ? 7000 : 2500;
  const double slower = f32 ? (ks ? 1.5 : 1) : edge ? 2 : 1;
  const long most_ns = !copies ? 17000 : !ks ? 24000 : f32 ? 42000 : 35000;
  if (fixed + ns * slower <= (double)most_ns * units / blocks) return 1;
  const long tiles = (long)groups * ((m + 255) / 256), most = copies || tiles * 4 <= units ? 48 : ks ? 16 : 24;
  return n <= most * groups ? 1 : 0;
}

// counted with the smallest tiles any variant uses
bool grouped_n_fits(const Grouped16& g) {
  return group_tiles_max(g.n, g.groups, 32) * ((g.m + 15) / 16) <= 0x7fffffffL;  // (parts only where tiles are few)
}

// Parts of an inner dimension of `slices` slices for `tiles` tiles whose result
// has `entries` entries, from modelled times in us: rounds of whole tiles at
// 1.4 per slice and 9 besides (f32: 1.2 and 8), a last one of quarters at 0.6
// and 6 where it is at most half full (share.h), and the sums' way through
// memory at 4 TB/s and a launch.  Measured in us, the rule before (as many parts as quarters had
// units) / this: outer products of 32768 rows, bf16 1 of 2048 x 2048 555 / 247,
// 1 of 1024 x 1024 157 / 96, f32 1 of 1024 x 1024 860 / 388 (slices: 230).
static int parts_for(bool f32, long tiles, long slices, double entries) {
  const long units = 256;
  auto time = [&](long parts) {
    const long total = tiles * parts, rest = total % units;
    const double k = ceil((double)slices / parts);
    const double whole = f32 ? 1.2 * k + 8 : 1.4 * k + 9, quarter = (f32 ? 0.55 : 0.6) * k + 6;
    const double last = rest == 0 ? 0 : rest * 2 <= units ? quarter * ((4 * rest + units - 1) / units) : whole;
    return (total / units) * whole + last + (parts > 1 ? 8 + 2 * 4 * entries * parts / 4e6 : 0);
  };
  int best = 1;
  double least = 0.95 * time(1);
  for (int parts = 2; parts <= 32 && parts * tiles <= 2 * units && parts * 4 <= slices; ++parts)
    if (time(parts) < least) least = time(best = parts);
  return best;
}

int outer_parts(bool f32, int groups, int m, int q, int n) {
  const long tile = f32 ? 128 : 256;
  return parts_for(f32, ((m + tile - 1) / tile) * ((q + tile - 1) / tile) * groups,
                   ((long)n / groups + BK16 - 1) / BK16, (double)groups * m * q);
}

// Measured in us (the kernel for small outer products / tiles): its time is
// that of its 64 x 64 tiles' columns, 2^20 of them 30 us in 16 bits, 45 to 75
// off the 8-byte grid, 105 in f32, and 4 for each block on a unit, to look up,
// to start and to add; the tiles take a launch of each copy, exponent and sum
// in parts besides their own.
//   16-bit   8 of 256 x 256, 4096 rows 7 / 9, 32768 25 / 21;  16 of 512 x 512, 4096 rows 18 / 10
//   copied   8 of 255 x 255, 4096 rows 10 / 26;  1 of 1023 x 1023, 4096 rows 57 / 39
//   f32      8 of 256 x 256, 4096 rows 15 / 40;  1 of 1024 x 1024, 4096 rows 104 / 77
int few_outer_parts(bool f32, bool edge, int groups, int m, int q, int n) {
  const long blocks = few_outer_blocks(groups, m, q), each = std::max(((long)n + groups - 1) / groups, 1L);
  if (blocks > std::min((f32 || edge ? 1L << 19 : 1L << 18) / each, f32 ? 1536L : 512L)) return 0;
  const long chunks = (each + (f32 ? 127 : 255)) / (f32 ? 128 : 256);
  return (int)std::max(std::min({512 / blocks, chunks / 4, 32L}), 1L);
}

size_t outer_partial_bytes(int parts, int groups, int m, int q) {
  return parts > 1 ? (size_t)parts * groups * m * q * 4 : 0;
}

int gemm_parts(bool f32, int groups, int m, int n, int q) {
  const long tile = f32 ? 128 : 256;
  return parts_for(f32, group_tiles_max(n, groups, tile) * ((m + tile - 1) / tile), (q + BK16 - 1) / BK16,
                   (double)m * n);
}

size_t gemm_partial_bytes(int parts, int m, int n) { return parts > 1 ? (size_t)parts * m * n * 4 : 0; }

bool grouped_k_fits(const Grouped16& g) {
  return (long)((g.m + 63) / 64) * ((g.q + 63) / 64) <= 0x7fffffffL / g.groups;
}

hipError_t launch_grouped_n(const Grouped16& g, hipStream_t st) {
  if (g.few) return g.f32 ? few<Single>(g, st) : g.bf16 ? few<Bfloat>(g, st) : few<Half>(g, st);
  if (g.B.ks || (g.f32 && g.A.ks)) return hipErrorInvalidValue;
  if (g.f32) return grouped_n<Half, 128, false, true>(g, st);
  if (g.bf16) return g.A.ks ? grouped_n<Bfloat, 256, true, false>(g, st) : grouped_n<Bfloat, 256, false, false>(g, st);
  return g.A.ks ? grouped_n<Half, 256, true, false>(g, st) : grouped_n<Half, 256, false, false>(g, st);
}

hipError_t launch_grouped_k(const Grouped16& g, hipStream_t st) {
  if (g.few) return g.f32 ? few_outer<Single>(g, st) : g.bf16 ? few_outer<Bfloat>(g, st) : few_outer<Half>(g, st);
  if (g.A.ks != g.B.ks || (g.f32 && g.A.ks)) return hipErrorInvalidValue;
  if (g.f32) return grouped_k<Half, 128, false, true>(g, st);
  if (g.bf16) return g.A.ks ? grouped_k<Bfloat, 256, true, false>(g, st) : grouped_k<Bfloat, 256, false, false>(g, st);
  return g.A.ks ? grouped_k<Half, 256, true, false>(g, st) : grouped_k<Half, 256, false, false>(g, st);
}

}  // namespace oz
