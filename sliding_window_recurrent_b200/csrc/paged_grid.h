// Sizes of the paged decode step's grid, from the descriptor alone: host arithmetic
// without CUDA, so that it can be checked where there is no GPU.
#pragma once

#include <cstdint>

namespace maglev {

constexpr int KSTEP = 16;  // keys of a step
// A unit counts as this many steps more than it has: its query, its new entry and
// its end keep a warp from its copies for about that time, and a warp dealt only
// short units ended last (64 sequences of 64 to 4096: 108 us, 96 on average; 512
// of up to 190: 72, 66, 61, 61 us in all with 1, 2, 3, 4).
constexpr int UNIT_COST = 3;

// Blocks of `teams` teams for B sequences of `units` units each: as many as the GPU
// holds at once (`resident`), fewer where there cannot be that many steps. Never more
// than `resident`: the workspace has room for the parts of that many blocks' teams.
inline int64_t decode_blocks(int B, int units, int max_pages, int page_size, int window, int teams, int64_t resident) {
  int64_t keys = (int64_t)max_pages * page_size;
  // a window may be any int: in 32 bits the sum wraps from 2^31 - 16 on, and the grid with it
  if (window > 0 && (int64_t)window + KSTEP < keys) keys = (int64_t)window + KSTEP;
  const int64_t steps = ((keys + KSTEP - 1) / KSTEP + UNIT_COST) * units * B;
  const int64_t most = (steps + teams - 1) / teams;  // a step each
  const int64_t blocks = resident < most ? resident : most;
  return blocks < 1 ? 1 : blocks;
}

}  // namespace maglev
