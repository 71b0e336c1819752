// Launches of more blocks than one may have (host code; a CPU test driver
// builds it too).
#pragma once

namespace oz {

// A launch has fewer than 2^32 threads along a dimension of its grid: with up
// to 512 in a block, 2^22 blocks are well inside.
constexpr long PIECE_BLOCKS = 1L << 22;

// launch(first, count) for consecutive runs of at most PIECE_BLOCKS of `blocks`
// blocks: nearly always one.
template <class Launch>
void in_pieces(long blocks, Launch launch) {
  for (long first = 0; first < blocks; first += PIECE_BLOCKS)
    launch(first, (unsigned)(blocks - first < PIECE_BLOCKS ? blocks - first : PIECE_BLOCKS));
}

}  // namespace oz
