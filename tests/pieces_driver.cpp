// The pieces of launches of many sizes: argument by argument, the number of
// pieces, whether they follow one another from 0 to the last block, and the
// largest number of blocks of one.
#include <cstdio>
#include <cstdlib>

#include "../fp64_gemm_emulation_ozii_amd/csrc/pieces.h"

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    const long blocks = std::atol(argv[i]);
    long next = 0, most = 0, pieces = 0;
    bool whole = true;
    oz::in_pieces(blocks, [&](long first, unsigned count) {
      whole = whole && first == next && count > 0;
      next = first + (long)count;
      most = (long)count > most ? (long)count : most;
      ++pieces;
    });
    std::printf("%ld %d %ld\n", pieces, (int)(whole && next == blocks), most);
  }
  return 0;
}
