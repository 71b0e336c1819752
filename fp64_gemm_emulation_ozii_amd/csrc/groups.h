// Ragged groups on the device: where the group tiles of a launch lie.
//
// J_e = [offsets[e], offsets[e + 1]) for e < groups, read on the device so
// that a call never waits for them.  The boundaries used are
//   b_0 = clamp(offsets[0]),  b_e = max(b_{e-1}, clamp(offsets[e])),
// clamp to [0, n]: for offsets in order they are the offsets, and for any
// others the groups stay disjoint and inside [0, n], so no launch bound and
// no buffer size can be passed whatever the offsets hold.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace oz {

// Tiles of `tile` entries that groups of n entries in all can need:
// sum ceil(len_e / tile) <= (n + groups (tile - 1)) / tile, and at most one
// group more than n can hold entries.
inline long group_tiles_max(long n, long groups, long tile) {
  const long nonempty = groups < n ? groups : n;
  return (n + nonempty * (tile - 1)) / tile;
}

struct GroupTile {
  int group;    // -1: no such tile
  int begin;    // first entry of the tile
  int end;      // end of the group
  int tile;     // the tile's place in its group
  int first;    // tiles of all groups before this one
};

__device__ __forceinline__ int wave_scan_max(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v = v > o ? v : o;
  }
  return v;
}

__device__ __forceinline__ int wave_scan_add(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}

// One wavefront walks the groups 64 at a time: lane l holds group e0 + l's
// boundaries and the tiles up to and with it.  visit(e0, begin, end, upto)
// returns true to stop; the tiles of all groups walked come back.
template <class Visit>
__device__ __forceinline__ int walk_groups(const int32_t* __restrict__ offsets, int groups, int n, int tile,
                                           Visit visit) {
  const int lane = threadIdx.x & 63;
  int carry = 0;  // tiles of the groups before e0
  int bound = min(max(offsets[0], 0), n);
  for (int e0 = 0; e0 < groups; e0 += 64) {
    const int e = e0 + lane;
    int hi = e < groups ? min(max(offsets[e + 1], 0), n) : 0;
    hi = max(wave_scan_max(hi), bound);
    int lo = __shfl_up(hi, 1);
    if (lane == 0) lo = bound;
    const int upto = carry + wave_scan_add(e < groups ? (hi - lo + tile - 1) / tile : 0);
    if (visit(e0, lo, hi, upto)) return upto;
    bound = __builtin_amdgcn_readlane(hi, 63);
    carry = __builtin_amdgcn_readlane(upto, 63);
  }
  return carry;
}

// The tile number idx in the order of the groups (called by whole
// wavefronts; every lane gets the same answer).
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* __restrict__ offsets, int groups, int n, int tile,
                                                     int idx) {
  GroupTile t{-1, 0, 0, 0, 0};
  walk_groups(offsets, groups, n, tile, [&](int e0, int lo, int hi, int upto) {
    const unsigned long long over = __ballot(upto > idx);
    if (over == 0) return false;
    const int l = __ffsll((unsigned long long)over) - 1;
    const int begin = __builtin_amdgcn_readlane(lo, l);
    const int count = (__builtin_amdgcn_readlane(hi, l) - begin + tile - 1) / tile;
    t.group = e0 + l;
    t.end = __builtin_amdgcn_readlane(hi, l);
    t.first = __builtin_amdgcn_readlane(upto, l) - count;
    t.tile = idx - t.first;
    t.begin = begin + t.tile * tile;
    return true;
  });
  return t;
}

// Group e's boundaries and the tiles of the groups before it.
__device__ __forceinline__ GroupTile group_at(const int32_t* __restrict__ offsets, int groups, int n, int tile,
                                              int e) {
  GroupTile t{-1, 0, 0, 0, 0};
  walk_groups(offsets, groups, n, tile, [&](int e0, int lo, int hi, int upto) {
    if (e >= e0 + 64) return false;
    const int l = e - e0;
    t.group = e;
    t.begin = __builtin_amdgcn_readlane(lo, l);
    t.end = __builtin_amdgcn_readlane(hi, l);
    t.first = __builtin_amdgcn_readlane(upto, l) - (t.end - t.begin + tile - 1) / tile;
    return true;
  });
  return t;
}

// The groups' tiles for a wavefront that looks up many: up to 64 groups are
// walked once and kept, one per lane.
struct GroupIndex {
  const int32_t* offsets;
  int groups, n, tile;
  int lo, hi, upto;  // lane l: group l (groups <= 64)
  int total;

  __device__ __forceinline__ GroupIndex(const int32_t* o, int g, int nn, int t) : offsets(o), groups(g), n(nn), tile(t) {
    total = __builtin_amdgcn_readfirstlane(walk_groups(offsets, groups, n, tile, [&](int, int l, int h, int u) {
      lo = l;
      hi = h;
      upto = u;
      return false;
    }));
  }

  __device__ __forceinline__ GroupTile find(int idx) const {
    if (groups > 64) return find_group_tile(offsets, groups, n, tile, idx);
    GroupTile t{-1, 0, 0, 0, 0};
    const unsigned long long over = __ballot(upto > idx);
    if (over == 0) return t;
    const int l = __ffsll(over) - 1;
    t.group = l;
    t.end = __builtin_amdgcn_readlane(hi, l);
    const int begin = __builtin_amdgcn_readlane(lo, l);
    t.first = __builtin_amdgcn_readlane(upto, l) - (t.end - begin + tile - 1) / tile;
    t.tile = idx - t.first;
    t.begin = begin + t.tile * tile;
    return t;
  }

  // Group e's boundaries and the tiles of the groups before it.
  __device__ __forceinline__ GroupTile at(int e) const {
    if (groups > 64) return group_at(offsets, groups, n, tile, e);
    GroupTile t{e, 0, 0, 0, 0};
    t.begin = __builtin_amdgcn_readlane(lo, e);
    t.end = __builtin_amdgcn_readlane(hi, e);
    t.first = __builtin_amdgcn_readlane(upto, e) - (t.end - t.begin + tile - 1) / tile;
    return t;
  }
};

}  // namespace oz
