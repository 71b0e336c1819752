// How the blocks of a grouped product share its tiles out (host and device
// code; a CPU test driver builds it too).
#pragma once

#ifndef __HIPCC__
#ifndef __host__
#define __host__
#endif
#ifndef __device__
#define __device__
#endif
#ifndef __forceinline__
#define __forceinline__ inline
#endif
#endif

namespace oz {

// `total` tiles on `units` compute units, which run one block each at a time,
// in SHARES units blocks.  The first `units` blocks walk whole rounds of
// tiles; the last full round goes to the next `units` blocks, one tile each
// as units become free (tiles at the end of a group are cheaper than others);
// what then remains is less than a round, and where it is no more than half
// of one, its tiles are cut into quarters for the last 2 units blocks, or else
// taken whole.
constexpr int SHARES = 4;

struct Share {
  int rounds;   // tiles first, first + units, ... of this block
  int first;    // -1: none
  int quarter;  // -1: whole tiles; else that quarter of tile `first`
};

__host__ __device__ __forceinline__ Share share_of(int total, int units, int block) {
  const int rounds = total / units > 1 ? total / units - 1 : 0;
  const int kept = rounds * units;
  if (block < units) return Share{rounds, rounds > 0 ? block : -1, -1};
  block -= units;
  const int left = total - kept;  // less than two rounds
  const int full = left >= units ? units : 0;
  if (block < units) return Share{1, block < full ? kept + block : -1, -1};
  block -= units;
  const int rest = left - full;
  if (rest * 2 <= units) return Share{1, block < rest * 4 ? kept + full + block / 4 : -1, block % 4};
  return Share{1, block < rest ? kept + full + block : -1, -1};
}

// Blocks that a launch of at most `most` tiles can leave out from the first
// on: those without a share whatever the tiles are (a block without one still
// waits for a unit and looks the tiles up: 2 us each).
inline int shares_without(long most, int units) { return most < units ? 2 * units : most < 2L * units ? units : 0; }

}  // namespace oz
