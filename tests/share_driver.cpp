// Walks the shares of every block and counts how often each quarter of each
// tile is taken.  Arguments: units, largest total.  Prints the first fault or
// "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../fp64_gemm_emulation_ozii_amd/csrc/share.h"

int main(int argc, char** argv) {
  const int units = std::atoi(argv[1]), most = std::atoi(argv[2]);
  (void)argc;
  for (int total = 0; total <= most; ++total) {
    std::vector<int> seen(4 * (size_t)total, 0);
    for (int block = 0; block < oz::SHARES * units; ++block) {
      const oz::Share s = oz::share_of(total, units, block);
      if (s.first < 0) continue;
      if (block < oz::shares_without(total, units)) {
        std::printf("units %d total %d block %d: left out, but has tile %d\n", units, total, block, s.first);
        return 1;
      }
      for (int r = 0; r < (s.quarter >= 0 ? 1 : s.rounds); ++r) {
        const long tile = s.first + (long)r * units;
        if (tile < 0 || tile >= total) {
          std::printf("units %d total %d block %d: tile %ld\n", units, total, block, tile);
          return 1;
        }
        for (int q = 0; q < 4; ++q)
          if (s.quarter < 0 || s.quarter == q) ++seen[4 * tile + q];
      }
    }
    for (size_t i = 0; i < seen.size(); ++i)
      if (seen[i] != 1) {
        std::printf("units %d total %d: quarter %zu of tile %zu taken %d times\n", units, total, i % 4, i / 4, seen[i]);
        return 1;
      }
  }
  std::printf("ok\n");
  return 0;
}
