// Products of 8-bit operands in scaled blocks (gemm8.h) on gfx950 matrix cores.
//
// Two ways to sum a block's 128 products:
//   narrow  one v_mfma_f32_16x16x128_f8f6f4, for results of 16 bits and more than 16 columns.  Within the
//           32 products that one lane holds the matrix core keeps what lies above
//           2^-13 of the largest.  Results of gaussian entries come out with an
//           error of 1.5e-5 of their norm, 4.6e-5 where one column in a hundred is 21 times
//           larger and 8.6e-5 where it is 301 times: a fourteenth, a fifth and two
//           fifths of float16's rounding (2.1e-4), and at most a twentieth of bfloat16's.  A single
//           result whose products cancel may be off by more of itself: half the time of the
//           wide products is what that buys, and float32 results are there for who needs them.
//   wide    four v_mfma_f32_16x16x32_f16 of the same entries as half precision
//           (both 8-bit types are exact there), for float32 results, whose sums are
//           float32 throughout, at half the rate; and for 16 columns and fewer, where
//           the weights' bytes count and not the products.
// A block's sum is then multiplied by its scales and added to the accumulators
// in float32.
#include <algorithm>
#include <atomic>

#include "block8.h"
#include "gemm8.h"
#include "products.h"
#include "tile16.h"

namespace oz {
namespace {

// x rounded to a 16-bit type, to nearest-even.
__device__ __forceinline__ uint16_t round16(float x, int ctype) {
  return ctype == OZGEMM_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
                              : __builtin_bit_cast(uint16_t, (_Float16)x);
}

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

// A block's sums of 16 x 16 results, of one fragment of A with G of B: lane l
// has rows 4 (l / 16) .. + 3 of column l mod 16.
template <int TA, int TB, bool WIDE, int G>
__device__ __forceinline__ void block_products(v4f (&d)[G], const Frag<TA, WIDE>& a, const Frag<TB, WIDE>* b) {
#pragma unroll
  for (int u = 0; u < G; ++u) d[u] = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (WIDE) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < G; ++u) d[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[t], b[u].h[t], d[u], 0, 0, 0);
  } else {
#pragma unroll
    for (int u = 0; u < G; ++u)  // (scales of 0 within the instruction: none)
      d[u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.w, b[u].w, d[u], TA == OZGEMM_E5M2, TB == OZGEMM_E5M2,
                                                              0, 0, 0, 0);
  }
}

__device__ __forceinline__ void pin(v4f& v) { asm volatile("" : "+v"(v)); }

// A mask of the bytes of a 16-byte piece before `left`.
__device__ __forceinline__ v4u8 first_bytes(int left) {
  v4u8 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int bits = min(max(left - 4 * k, 0), 4) * 8;
    v[k] = bits == 32 ? ~0u : (1u << bits) - 1u;
  }
  return v;
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------

// BM x BN results by WM x WN wavefronts, a block per compute unit that walks its
// tiles.  Blocks of 128 entries ("slices") go from HBM straight into LDS through two
// buffers, 16 bytes per lane, range-checked (rows past the end arrive as zeros, as do
// pieces past the inner dimension), with their rows' scales beside them.
//
// Two wavefronts share a SIMD, and each alternates one product with the scaling
// of the one before last: a wavefront alone takes 49 cycles for a product of 32 and its
// four multiply-adds, two together 38 each.  So nothing may hold both up:
// fragments are read from LDS a row of products ahead, those of B for the next slice
// right after their last use, and one barrier per slice stands before its last row:
// every wavefront has then read the slice, whose buffer the loads of the slice
// after the next go to, and the next slice, asked for a slice's time ago, has landed.
// The stream of slices runs on over the tiles' ends.
//
// Measured: 8192 x 8192 x 4096 narrow 251 to 322 us over twenty calls in a row (290 on average: the clock
// gives way to the power), 255 over four, the matrix cores busy for 51% of the cycles at 2.0 GHz.
// Of a wavefront's cycles 38% issue, 32% wait for an issue slot and 30% for loads, LDS or the barrier; of
// its 390 instructions a slice 32 are products, 179 others of the vector units, 91 scalar.
// 4096 x 4096 x 8192 wide 290 to 363 us with scales for every row of both (twenty calls; 284 in a shorter run,
// and 239 there where 128 rows share one): the conversions to half precision and the scaling take more issue slots than
// the products.  Accumulating by the scaled form of the instruction (for scales that are
// powers of two) took 6% less at best, two groups of wavefronts in turn at
// products and scaling more than this.
template <int TA, int TB, bool WIDE, bool AROW, int BM, int BN, int WM, int WN>
struct Tile8 {
  static constexpr int NW = WM * WN, THREADS = NW * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int ROWS = BM + BN;
  static constexpr int BUF = ROWS * 128, SLOT = THREADS * 4;  // of a slice; of its scales
  static constexpr int SMEM = 2 * (BUF + SLOT);
  static constexpr int LA = BM * 128 / 1024 / NW, LB = BN * 128 / 1024 / NW, LOADS = LA + LB + 1;  // of a wavefront
  static_assert(LA % 2 == 0 && LA * NW * 1024 == BM * 128, "whole wave loads, the first of an even number");
  static_assert(LB % 2 == 0 && LB * NW * 1024 == BN * 128, "whole wave loads, the first of an even number");
  static_assert(ROWS <= THREADS && BM % 64 == 0, "a scale and a row a thread");
  static_assert(FM % 4 == 0, "fragments of A and their scales change places, and stores take two");
  static __device__ __forceinline__ int swz(int row) { return ((row >> 1) ^ (row << 2)) & 7; }

  // A tile of the call: rows from m0 and n0 on, part `part`, entries k0 .. k_end.
  struct Place {
    int m0, n0, part, k0, k_end;
  };
  static __device__ __forceinline__ Place place(const Scaled8& g, int tile) {
    const int tiles_m = (g.m + BM - 1) / BM, tiles_n = (g.n + BN - 1) / BN, whole = tiles_m * tiles_n;
    Place p;
    p.part = tile / whole;
    int nj, mi;
    panel_order<4>(xcd_order(tile - p.part * whole, whole), tiles_n, tiles_m, nj, mi);
    p.m0 = __builtin_amdgcn_readfirstlane(mi * BM);
    p.n0 = __builtin_amdgcn_readfirstlane(nj * BN);
    p.part = __builtin_amdgcn_readfirstlane(p.part);
    const int each = (((g.q + 127) >> 7) + g.parts - 1) / g.parts * 128;
    p.k0 = __builtin_amdgcn_readfirstlane(p.part * each);
    p.k_end = __builtin_amdgcn_readfirstlane(min(g.q, p.k0 + each));
    return p;
  }

  // The loads of a block's slices, in order.
  struct Feed {
    const Scaled8& g;
    char* smem;
    int lane, wave, tile, tiles;
    const uint8_t *pa, *pb;
    const float* ps;
    long sstep;
    // This lane's row and piece of eight rows that begin at an even or an odd
    // multiple of 8: bytes from their first row, entries (one past the end: the
    // offset lies past it too).
    int kin0, kin1, offa0, offa1, offb0, offb1;
    int reca, recb;  // bytes from pa, pb to the end of the last row's last 16-byte piece
    int left;        // entries from the slice to load on
    int s;           // its number

    __device__ __forceinline__ Feed(const Scaled8& g_, char* lds, int lane_, int wave_, int tiles_)
        : g(g_), smem(lds), lane(lane_), wave(wave_), tile(blockIdx.x), tiles(tiles_), s(0) {
      kin0 = ((lane & 7) ^ swz(lane >> 3)) * 16;
      kin1 = ((lane & 7) ^ swz(8 + (lane >> 3))) * 16;
      begin();
    }
    __device__ __forceinline__ void begin() {
      const Place p = place(g, tile);
      pa = g.A.p + (long)p.m0 * g.A.ld + p.k0;
      pb = g.B.p + (long)p.n0 * g.B.ld + p.k0;
      const int len = (g.q + 15) / 16 * 16 - p.k0;
      reca = (min(g.m - p.m0, BM) - 1) * (int)g.A.ld + len;
      recb = (min(g.n - p.n0, BN) - 1) * (int)g.B.ld + len;
      const int first = wave * 64;
      const bool a = first < BM;
      const int row = a ? min(p.m0 + first + lane, g.m - 1) >> g.A.shift : min(p.n0 + first + lane - BM, g.n - 1);
      sstep = a ? g.A.sblock : g.B.sblock;
      ps = (a ? g.A.s + row * g.A.srow : g.B.s + row * g.B.srow) + (p.k0 >> 7) * sstep;
      left = p.k_end - p.k0;
      edge();
      uniform();
    }
    // What is the same in all lanes stays in scalar registers, as the loads need it.
    __device__ __forceinline__ void uniform() {
      pa = same(pa);
      pb = same(pb);
      reca = __builtin_amdgcn_readfirstlane(reca);
      recb = __builtin_amdgcn_readfirstlane(recb);
      left = __builtin_amdgcn_readfirstlane(left);
      tile = __builtin_amdgcn_readfirstlane(tile);
      s = __builtin_amdgcn_readfirstlane(s);
    }
    static __device__ __forceinline__ const uint8_t* same(const uint8_t* p) {
      const uint64_t u = (uint64_t)p;
      return (const uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)u) |
                              (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32);
    }
    __device__ __forceinline__ void edge() {
      const int r = lane >> 3, a = r * (int)g.A.ld, b = r * (int)g.B.ld, past = (int)0x80000000;
      offa0 = kin0 < left ? a + kin0 : past;
      offa1 = kin1 < left ? a + kin1 : past;
      offb0 = kin0 < left ? b + kin0 : past;
      offb1 = kin1 < left ? b + kin1 : past;
    }
    // 8 rows of an operand, `at` from its first, to where they lie in the buffer
    static __device__ __forceinline__ void rows8(const uint8_t* p, int records, int at, char* to) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, records, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, at, 0, 0, 0);
    }
    // load li of the slice
    __device__ __forceinline__ void load1(int li) const {
      char* to = smem + (s & 1) * (BUF + SLOT);
      if (li < LA) {
        const int row0 = (wave * LA + li) * 8;
        rows8(pa, reca, (li & 1 ? offa1 : offa0) + row0 * (int)g.A.ld, to + row0 * 128);
      } else if (li < LA + LB) {
        const int row0 = (wave * LB + li - LA) * 8;
        rows8(pb, recb, ((li - LA) & 1 ? offb1 : offb0) + row0 * (int)g.B.ld, to + (BM + row0) * 128);
      } else {
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)ps,
                                         (__attribute__((address_space(3))) void*)(to + BUF + wave * 256), 4, 0, 0);
      }
    }
    __device__ __forceinline__ void next() {
      ++s;
      left -= 128;
      if (left > 0) {
        pa += 128;
        pb += 128;
        reca -= 128;
        recb -= 128;
        ps += sstep;
        if (left < 128) edge();
      } else {
        tile += gridDim.x;
        if (tile < tiles)
          begin();
        else  // past the end: the loads go on, of zeros, for the counter's sake
          reca = recb = left = 0;
      }
      uniform();
    }
    __device__ __forceinline__ void all() {
#pragma unroll
      for (int li = 0; li < LOADS; ++li) load1(li);
      next();
    }
  };

  // The restrict-qualified argument gives the read an alias scope; without one
  // the compiler takes it to depend on the loads into LDS in flight.
  template <class V>
  static __device__ __forceinline__ V read(const char* __restrict__ p) {
    return *reinterpret_cast<const V*>(p);
  }

  // A slice has landed; of the last 16-byte piece of its rows `tail` bytes count, the others go.
  static __device__ __forceinline__ void arrive(char* buf, int left, int tail) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (left > 128 || tail == 0) return;
    const int r = threadIdx.x;
    if (r < ROWS) {
      v4u8* at = reinterpret_cast<v4u8*>(buf + r * 128 + (((left - 1) >> 4) ^ swz(r)) * 16);
      *at &= first_bytes(tail);
    }
    __syncthreads();
  }

  static constexpr int STORES = FM * FN / 2;

  static __device__ __forceinline__ void walk(const Scaled8& g, char* smem, int lane, int wave, int tiles) {
    const int wm = wave % WM, wn = wave / WM;
    Feed feed(g, smem, lane, wave, tiles);
    // rows 16 apart lie alike
    const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ swz(lane & 15)) * 16), at1 = at0 ^ 64;
    const int a_at = wm * (BM / WM) * 128, b_at = (BM + wn * (BN / WN)) * 128;
    const int sa_at = BUF + (wm * (BM / WM) + (AROW ? 4 * (lane >> 4) : 0)) * 4;
    const int sb_at = BUF + (BM + wn * (BN / WN) + (lane & 15)) * 4;
    v4u8 ra[2][2], rb[FN][2];
    v4f s4[4];
    float xn[FN], fn = 0.f;
    auto read_a = [&](const char* buf, int i) {
      ra[i & 1][0] = read<v4u8>(buf + a_at + i % FM * 2048 + at0);
      ra[i & 1][1] = read<v4u8>(buf + a_at + i % FM * 2048 + at1);
      if (AROW) s4[i & 3] = read<v4f>(buf + sa_at + i % FM * 64);
    };
    auto read_b = [&](const char* buf, int j) {
      rb[j][0] = read<v4u8>(buf + b_at + j * 2048 + at0);
      rb[j][1] = read<v4u8>(buf + b_at + j * 2048 + at1);
      xn[j] = read<float>(buf + sb_at + j * 64);
      if (!AROW && j == 0) fn = read<float>(buf + sa_at);
    };

    Place p = place(g, blockIdx.x);
    feed.all();
    feed.all();
    wait_loads<LOADS>();
    arrive(smem, p.k_end - p.k0, (p.k_end - p.k0) & 15);
    read_a(smem, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_b(smem, j);

    v4f acc[FM][FN];
    int s = 0, stored = 0;
    for (int tile = blockIdx.x; tile < tiles;) {
      const int next_tile = tile + gridDim.x;
      const Place then = next_tile < tiles ? place(g, next_tile) : p;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
          pin(acc[i][j]);  // (no copy of the loop for a first slice added to zeros)
        }
      for (int left = p.k_end - p.k0; left > 0; left -= 128, ++s) {
        char* buf = smem + (s & 1) * (BUF + SLOT);
        char* other = smem + (~s & 1) * (BUF + SLOT);
        Frag<TB, WIDE> b[FN];
        float xb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) xb[j] = AROW ? xn[j] : xn[j] * fn;
        // One or (wide) two products a slot, DELAY slots ahead of their scaling.
        // pin() keeps both where they stand: the compiler would put every
        // product right before its use and wait for it there.
        constexpr int G = WIDE ? 2 : 1, PER = FN / G, SLOTS = FM * PER, DELAY = WIDE ? 1 : 2;
        static_assert(FN % G == 0, "whole slots");
        v4f d[DELAY + 1][G];
        Frag<TA, WIDE> a;
#pragma unroll
        for (int r = 0; r < SLOTS + DELAY; ++r) {
          if (r < SLOTS) {
            const int i = r / PER;
            if (r % PER == 0) {
              a.set(ra[i & 1][0], ra[i & 1][1]);
              if (i < FM - 1) {
                read_a(buf, i + 1);
              } else {
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wavefront has read the slice,
                if (stored == STORES)                // and its loads of the next one have landed
                  wait_loads<STORES>();
                else
                  wait_loads<0>();
                const Place& q = left > 128 ? p : then;
                const int whole = q.k_end - q.k0;
                arrive(other, left > 128 ? left - 128 : whole, whole & 15);
                read_a(other, FM);
              }
            }
#pragma unroll
            for (int u = 0; u < G; ++u)
              if (i == 0) b[r % PER * G + u].set(rb[r % PER * G + u][0], rb[r % PER * G + u][1]);
            block_products<TA, TB, WIDE, G>(d[r % (DELAY + 1)], a, &b[r % PER * G]);
#pragma unroll
            for (int u = 0; u < G; ++u) pin(d[r % (DELAY + 1)][u]);
            if (i == FM - 1) {
#pragma unroll
              for (int u = 0; u < G; ++u) read_b(other, r % PER * G + u);
#pragma unroll
              for (int li = 0; li < LOADS; ++li)
                if (li * PER / LOADS == r % PER) feed.load1(li);
            }
          }
          if (r >= DELAY) {
            const int i = (r - DELAY) / PER;
#pragma unroll
            for (int u = 0; u < G; ++u) {
              const int j = (r - DELAY) % PER * G + u;
              v4f& from = d[(r - DELAY) % (DELAY + 1)][u];
              pin(from);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                acc[i][j][k] = __builtin_fmaf(from[k], AROW ? s4[i & 3][k] * xb[j] : xb[j], acc[i][j][k]);
              pin(acc[i][j]);
            }
          }
        }
        feed.next();
        stored = __builtin_amdgcn_readfirstlane(0);
        asm volatile("" : "+s"(stored));  // (no copy of the loop for the first slice)
      }
      stored = store(acc, g, p, lane, wm, wn);
      stored = __builtin_amdgcn_readfirstlane(stored);
      asm volatile("" : "+s"(stored));
      tile = next_tile;
      p = then;
    }
    wait_loads<0>();
  }

  // A tile's results, straight from the accumulators; how many stores every
  // wavefront of it is sure to have made (STORES, or 0 at the edges).  In 16 bits two
  // fragments' lanes swap halves, so that a lane writes 8 rows at once.
  static __device__ __forceinline__ int store(const v4f (&acc)[FM][FN], const Scaled8& g, const Place& p, int lane,
                                              int wm, int wn) {
    const int col0 = p.n0 + wn * (BN / WN) + (lane & 15), row0 = p.m0 + wm * (BM / WM);
    if (g.parts > 1 || g.ctype == OZGEMM_F32) {
      float* out = g.parts > 1 ? g.partial + (long)p.part * g.n * g.m : (float*)g.C;
      const long ld = g.parts > 1 ? g.m : g.ldc;
      const int row = row0 + 4 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if (col0 + j * 16 < g.n) {
          float* to = out + (col0 + j * 16) * ld + row;
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            if (row + i * 16 + 4 <= g.m) {
              *reinterpret_cast<v4f_any*>(to + i * 16) = acc[i][j];
            } else if (row + i * 16 < g.m) {
              some(to + i * 16, __builtin_bit_cast(v4u8, acc[i][j]), 4 * (g.m - row - i * 16));
            }
          }
        }
      }
      return 0;  // (twice as many as STORES)
    }
    const int row = row0 + ((lane >> 4) & 1) * 16 + 8 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      uint16_t* to = (uint16_t*)g.C + (long)(col0 + j * 16) * g.ldc + row;
#pragma unroll
      for (int i = 0; i < FM; i += 2) {
        uint32_t w[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w[u][k] = round16(acc[i + u][j][2 * k], g.ctype) | (uint32_t)round16(acc[i + u][j][2 * k + 1], g.ctype) << 16;
        // lanes 16 .. 31 and 48 .. 63 of the first for lanes 0 .. 15 and 32 .. 47 of the second: rows 0 .. 7 of
        // fragment i, then of i + 1, rows 8 .. 15 of i, then of i + 1
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const auto x = __builtin_amdgcn_permlane16_swap(w[0][k], w[1][k], false, false);
          w[0][k] = x[0];
          w[1][k] = x[1];
        }
        const v4u8 v = {w[0][0], w[0][1], w[1][0], w[1][1]};
        if (col0 + j * 16 < g.n) {
          if (row + i * 16 + 8 <= g.m)
            *reinterpret_cast<v4u_at2*>(to + i * 16) = v;
          else if (row + i * 16 < g.m)
            some(to + i * 16, v, 2 * (g.m - row - i * 16));
        }
      }
    }
    return p.m0 + BM <= g.m && p.n0 + BN <= g.n ? STORES : 0;
  }

  // The first bytes (a multiple of 2, under 16) of v; a loop, as code that few tiles run has to be fetched too.
  static __device__ __forceinline__ void some(void* to, v4u8 v, int bytes) {
    uint16_t* p = (uint16_t*)to;
#pragma unroll 1
    for (int k = 0; k < bytes; k += 2) {
      *p++ = (uint16_t)v[0];
      v = v4u8{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    }
  }
};

template <class Tile>
__global__ __launch_bounds__(Tile::THREADS) void scaled_tiles_kernel(Scaled8 g, int tiles) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tile::walk(g, smem, lane, wave, tiles);
}

// The sum of the parts, in their order: a block per column and 1024 rows.
__global__ __launch_bounds__(256) void join_parts_kernel(Scaled8 g, int parts) {
  const int row = blockIdx.y * 1024 + threadIdx.x * 4;
  const long col = blockIdx.x;
  if (row >= g.m) return;
  const v4f v = sum_parts(g.partial + col * g.m + row, (long)g.n * g.m, parts, g.m - row);
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
// Few columns, and few results of any shape
// ---------------------------------------------------------------------------

// Few columns are bound by reading A once, few results by the time from one slice to the
// next: a tile above takes 0.7 us for each, however small it is.  A block takes 16 RG rows
// and up to 16 FN columns; its eight wavefronts are RG of rows by KG of the inner dimension, of which
// KG blocks of 128 make a step.  A step's operands go to LDS through NB buffers, whole
// rows' 128 bytes by eight lanes each: read straight into MFMA operands, 16 neighbouring
// lanes would ask for 16 different lines (64 columns of 8192 x 4096: 19 us so, 15
// by way of LDS, both with wide products).  The KG sums meet in LDS, in a fixed order.
template <int TA, int TB, bool WIDE, bool AROW, int RG, int FN>
struct Few8 {
  static constexpr int KG = 8 / RG, COLS = 16 * FN, ROWS = RG + FN;  // sixteens of rows in a block's tile
  static constexpr int TILE = ROWS * 2048, STAGE = KG * TILE + 8 * 256;
  static constexpr int LOADS = ROWS * 2 / RG + 1;  // of a wavefront in a step
  static constexpr int NB = 150 * 1024 / STAGE < 4 ? 150 * 1024 / STAGE : 4;
  static constexpr int SUMS = KG * RG * FN * 1024;
  static constexpr int SMEM = NB * STAGE > SUMS ? NB * STAGE : SUMS;
  static_assert(ROWS * 2 % RG == 0 && NB >= 3, "whole wave loads, two steps ahead");
  static __device__ __forceinline__ int swz(int row) { return ((row >> 1) ^ (row << 2)) & 7; }
  template <class V>
  static __device__ __forceinline__ V read(const char* __restrict__ p) {
    return *reinterpret_cast<const V*>(p);
  }

  static __device__ __forceinline__ void run(const Scaled8& g, char* smem) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / RG, rg = wave % RG, m0 = blockIdx.x * 16 * RG, n0 = blockIdx.y * 16 * FN;
    const int steps = (((g.q + 127) >> 7) + KG - 1) / KG;
    // the loads of this wavefront's block, which its RG wavefronts share out
    const uint8_t* pa = g.A.p + (long)m0 * g.A.ld + kg * 128;
    const uint8_t* pb = g.B.p + (long)n0 * g.B.ld + kg * 128;
    const int len = (g.q + 15) / 16 * 16 - kg * 128;
    int reca = (min(g.m - m0, 16 * RG) - 1) * (int)g.A.ld + len, recb = (min(g.n - n0, 16 * FN) - 1) * (int)g.B.ld + len;
    const bool a = rg == 0;  // which scales
    const int srow = a ? min(m0 + lane, g.m - 1) >> g.A.shift : 0;
    const int scol = min(n0 + lane, g.n - 1);
    const int past = (g.q - 1) >> 7;  // the last block
    int issued = 0;
    auto issue = [&]() {
      const int k = (issued * KG + kg) * 128, left = g.q - k;
      char* to = smem + issued % NB * STAGE + kg * TILE;
#pragma unroll
      for (int li = 0; li < LOADS - 1; ++li) {
        const int idx = li * RG + rg, r = lane >> 3;
        const bool of_a = idx < RG * 2;
        const int row0 = of_a ? idx * 8 : (idx - RG * 2) * 8;
        const int kin = ((lane & 7) ^ swz((idx & 1) * 8 + r)) * 16;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(of_a ? pa : pb), 0, left > 0 ? (of_a ? reca : recb) : 0, 0x00020000);
        const int at = kin < left ? (row0 + r) * (int)(of_a ? g.A.ld : g.B.ld) + kin : (int)0x80000000;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(to + idx * 1024), 16, at,
                                                 0, 0, 0);
      }
      const int b = min(issued * KG + kg, past);
      const float* s = RG > 1 ? (a ? g.A.s + srow * g.A.srow + b * g.A.sblock : g.B.s + scol * g.B.srow + b * g.B.sblock)
                              : (lane < 32 ? g.A.s + (min(m0 + (lane & 15), g.m - 1) >> g.A.shift) * g.A.srow +
                                                 b * g.A.sblock
                                           : g.B.s + min(n0 + lane - 32, g.n - 1) * g.B.srow + b * g.B.sblock);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)s,
          (__attribute__((address_space(3))) void*)(smem + issued % NB * STAGE + KG * TILE + wave * 256), 4, 0, 0);
      ++issued;
      pa += KG * 128;
      pb += KG * 128;
      reca -= KG * 128;
      recb -= KG * 128;
    };
#pragma unroll
    for (int b = 0; b < NB - 1; ++b) issue();
    v4f acc[FN] = {};
    const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ swz(lane & 15)) * 16), at1 = at0 ^ 64;
    // where the two kinds of scales lie, from a block's first wavefront's place on
    const int sa_at = (AROW ? rg * 16 + 4 * (lane >> 4) : rg * 16) * 4, sb_at = (RG > 1 ? 64 : 32) * 4 + (lane & 15) * 4;
    for (int t = 0; t < steps; ++t) {
      slice_barrier<(NB - 2) * LOADS>();  // step t has landed, and everybody has read step t - 1
      issue();
      const char* tile = smem + t % NB * STAGE + kg * TILE;
      const char* scales = smem + t % NB * STAGE + KG * TILE + kg * RG * 256;
      v4u8 ra[2], rb[FN][2];
      ra[0] = read<v4u8>(tile + rg * 2048 + at0);
      ra[1] = read<v4u8>(tile + rg * 2048 + at1);
      float xb[FN];
      v4f s4;
      if (AROW)
        s4 = read<v4f>(scales + sa_at);
      else
        s4[0] = s4[1] = s4[2] = s4[3] = read<float>(scales + sa_at);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        rb[j][0] = read<v4u8>(tile + (RG + j) * 2048 + at0);
        rb[j][1] = read<v4u8>(tile + (RG + j) * 2048 + at1);
        xb[j] = read<float>(scales + sb_at + j * 64);
      }
      const int left = g.q - (t * KG + kg) * 128;
      if (left < 128 && (left & 15) != 0) {  // the rows' last piece ends inside it
        int have = left - (lane >> 4) * 16;
        asm volatile("" : "+v"(have));  // (the masks are worked out here, not in every step)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4u8 keep = first_bytes(have - h * 64);
          ra[h] &= keep;
#pragma unroll
          for (int j = 0; j < FN; ++j) rb[j][h] &= keep;
        }
      }
      Frag<TA, WIDE> fa;
      Frag<TB, WIDE> fb[FN];
      fa.set(ra[0], ra[1]);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j].set(rb[j][0], rb[j][1]);
      v4f d[FN];
      block_products<TA, TB, WIDE, FN>(d, fa, fb);
      if (left > 0) {  // (scales past the end may be anything)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[j][r] = __builtin_fmaf(d[j][r], s4[r] * xb[j], acc[j][r]);
      }
    }
    slice_barrier<0>();
    v4f* sums = reinterpret_cast<v4f*>(smem);
#pragma unroll
    for (int j = 0; j < FN; ++j) sums[(wave * FN + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int u = (int)threadIdx.x; u < RG * FN * 64; u += 512) {
      const int l = u & 63, j = u / 64 % FN, i = u / 64 / FN;
      v4f v = sums[(i * FN + j) * 64 + l];
#pragma unroll
      for (int w = 1; w < KG; ++w) v += sums[((w * RG + i) * FN + j) * 64 + l];
      const int col = n0 + j * 16 + (l & 15), row = m0 + i * 16 + 4 * (l >> 4);
      if (col >= g.n) continue;
      const long to = (long)col * g.ldc + row;
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
};

template <class Few>
__global__ __launch_bounds__(512) void scaled_few_kernel(Scaled8 g) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  Few::run(g, smem);
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

// A lane takes four blocks of a row, so that neighbouring lanes write next to each other.
__global__ __launch_bounds__(256) void turn_scales_kernel(const float* src, long srow, long sblock, int rows, int blocks,
                                                          float* dst) {
  const int r = blockIdx.x * 64 + (threadIdx.x & 63), b = (blockIdx.y * 4 + (threadIdx.x >> 6)) * 4;
  if (r >= rows) return;
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = src[r * srow + min(b + k, blocks - 1) * sblock];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (b + k < blocks) dst[(long)(b + k) * rows + r] = v[k];
}

constexpr int FEW8_COLS = 64;  // of one block

hipError_t join(const Scaled8& g, int parts, hipStream_t st) {
  join_parts_kernel<<<dim3(g.n, (g.m + 1023) / 1024), 256, 0, st>>>(g, parts);
  return hipGetLastError();
}

// Lets a kernel have that much LDS, once for every device (a bit each).
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& known) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (known.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) known.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int TA, int TB, bool WIDE, bool AROW, int BM, int BN, int WM>
hipError_t launch_tiles(const Scaled8& g, hipStream_t st) {
  using Tile = Tile8<TA, TB, WIDE, AROW, BM, BN, WM, 8 / WM>;
  const long tiles = (long)((g.m + BM - 1) / BM) * ((g.n + BN - 1) / BN) * g.parts;
  const long room = 256 * (160 * 1024 / Tile::SMEM);  // blocks that the card holds
  auto kernel = scaled_tiles_kernel<Tile>;
  static std::atomic<uint64_t> known{0};
  const hipError_t e = allow_lds((const void*)kernel, Tile::SMEM, known);
  if (e != hipSuccess) return e;
  kernel<<<(unsigned)std::min(tiles, room), Tile::THREADS, Tile::SMEM, st>>>(g, (int)tiles);
  return hipGetLastError();
}

template <class Few>
hipError_t few_kernel(const Scaled8& g, int rows, hipStream_t st) {
  auto kernel = scaled_few_kernel<Few>;
  static std::atomic<uint64_t> known{0};
  const hipError_t e = allow_lds((const void*)kernel, Few::SMEM, known);
  if (e != hipSuccess) return e;
  kernel<<<dim3((g.m + rows - 1) / rows, (g.n + Few::COLS - 1) / Few::COLS), 512, Few::SMEM, st>>>(g);
  return hipGetLastError();
}

// How a product is worked out.
enum class Way {
  FEW,     // up to 64 columns: blocks of 16 or 32 rows
  FEW32,   // blocks of 32 rows and 64 columns
  FEW64,   // blocks of 64 rows and 64 columns
  TILES,   // 128 x 128
  BIG,     // 256 x 256, wide products 256 x 128
};

// Above 64 columns: what takes the least time by measured costs, in us, where a unit is a
// block at once on each of the 256 compute units (TILES: two, the second one at 0.57).
//   FEW32   2 and, a round of units, 1.9 and 0.73 a step of four slices
//   FEW64   2 and 2.8 and 0.57 a step of two slices
//   TILES   3.3 and 0.72 a slice, 0.57 more for every further unit; for parts of the inner
//           dimension 4 and their sums written and read at 4 TB/s
//   BIG     5 and 1.8 a slice
// Measured, of 4096 x 4096, FEW32 / FEW64 / TILES / BIG: 128 columns 9.7 / 13.4 / 17.3 (4 parts) / 49,
// 200 of them 17.5 / 13.6 / 20 / 49, 512 of them 33 / 26 / 27 / 51; 2048 columns of 4096 x 4096
// 131 / 98 / 43 / 53; 1000 columns of 16384 x 4096 - / 209 / 86 / 62.
// Wide products take 1.5 to 1.9 times as long each way, so the choice is the same but for further
// units of TILES, which cost them as much as the first: 1000 columns of 8192 x 4096 81 by those, 63 by BIG.
Way way_of(int m, int n, int q, int* parts) {
  *parts = 1;
  if (n <= FEW8_COLS) return Way::FEW;
  const auto per = [](long a, long b) { return (a + b - 1) / b; };
  const auto units = [&](int rows, int cols, long p) { return (double)per(per(m, rows) * per(n, cols) * p, 256); };
  const long slices = per(q, 128);
  Way way = Way::FEW32;
  double best = 2.0 + units(32, 64, 1) * (1.9 + 0.73 * (double)per(slices, 4));
  const auto offer = [&](double t, Way w, long p) {
    if (t >= best) return;
    best = t;
    way = w;
    *parts = (int)p;
  };
  offer(2.0 + units(64, 64, 1) * (2.8 + 0.57 * (double)per(slices, 2)), Way::FEW64, 1);
  for (long p = 1; p <= 16 && p * 2 <= std::max(2L, slices); ++p) {
    const long each = per(slices, p);
    const double sums = p > 1 ? 4.0 + (double)p * m * n * 8.0 / 4e6 : 0.0;
    offer(3.3 + (0.15 + 0.57 * units(128, 128, p)) * (double)each + sums, Way::TILES, per(slices, each));  // (no empty part)
  }
  offer(5.0 + 1.8 * units(256, 256, 1) * (double)slices, Way::BIG, 1);
  return way;
}

// Few columns: 32 rows a block where that leaves a block for every compute unit, or where
// LDS has no room for the columns of eight blocks of the inner dimension.
template <int TA, int TB, bool WIDE, bool AROW>
hipError_t few_columns(const Scaled8& g, Way way, hipStream_t st) {
  const bool two = g.m >= 32 * 256;
  if (way == Way::FEW64) return few_kernel<Few8<TA, TB, WIDE, AROW, 4, 4>>(g, 64, st);
  if (g.n > 32) return few_kernel<Few8<TA, TB, WIDE, AROW, 2, 4>>(g, 32, st);
  return two ? few_kernel<Few8<TA, TB, WIDE, AROW, 2, 2>>(g, 32, st) : few_kernel<Few8<TA, TB, WIDE, AROW, 1, 2>>(g, 16, st);
}

template <int TA, int TB, bool AROW>
hipError_t launch_few(const Scaled8& g, Way way, hipStream_t st) {
  if (g.n <= 16)
    return g.m >= 32 * 256 ? few_kernel<Few8<TA, TB, true, AROW, 2, 1>>(g, 32, st)
                           : few_kernel<Few8<TA, TB, true, AROW, 1, 1>>(g, 16, st);
  return g.ctype == OZGEMM_F32 ? few_columns<TA, TB, true, AROW>(g, way, st) : few_columns<TA, TB, false, AROW>(g, way, st);
}

template <int TA, int TB, bool AROW>
hipError_t launch_kind(const Scaled8& g, hipStream_t st) {
  if (g.q == 0) return join(g, 0, st);
  int parts;
  const Way way = way_of(g.m, g.n, g.q, &parts);
  if (way <= Way::FEW64) return launch_few<TA, TB, AROW>(g, way, st);
  const bool wide = g.ctype == OZGEMM_F32;
  hipError_t e;
  // A second tile of a unit costs wide products as much as the first (way_of), so they go by the larger ones from there
  // on; scaled_big, which knows no type of results, does not say so, and their scales are read as they lie.
  const bool more = (long)((g.m + 127) / 128) * ((g.n + 127) / 128) > 256;
  if (way == Way::BIG || (wide && more && parts == 1))
    e = wide ? launch_tiles<TA, TB, true, AROW, 256, 128, 4>(g, st) : launch_tiles<TA, TB, false, AROW, 256, 256, 2>(g, st);
  else
    e = wide ? launch_tiles<TA, TB, true, AROW, 128, 128, 2>(g, st) : launch_tiles<TA, TB, false, AROW, 128, 128, 2>(g, st);
  return e != hipSuccess || g.parts == 1 ? e : join(g, g.parts, st);
}

template <int TA, int TB>
hipError_t launch_types(const Scaled8& g, hipStream_t st) {
  return g.A.shift == 0 ? launch_kind<TA, TB, true>(g, st) : launch_kind<TA, TB, false>(g, st);
}

}  // namespace

int scaled_parts(int m, int n, int q) {
  int parts;
  way_of(m, n, q, &parts);
  return parts;
}

bool scaled_big(int m, int n, int q) {
  int parts;
  return way_of(m, n, q, &parts) == Way::BIG;
}

hipError_t launch_turn_scales(const float* src, long srow, long sblock, int rows, int q, float* dst, hipStream_t st) {
  const int blocks = (q + 127) / 128;
  turn_scales_kernel<<<dim3((rows + 63) / 64, (blocks + 15) / 16), 256, 0, st>>>(src, srow, sblock, rows, blocks, dst);
  return hipGetLastError();
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
