// Grids of very many blocks (not installed).  An axis of a grid holds fewer than 2^32
// threads; one with more runs, without an error, what is left of them behind 32 bits.
#pragma once
#include <hip/hip_runtime.h>

namespace qmoe {

constexpr long long kGridX = 1 << 21;  // blocks along the first axis, of up to 1024 threads
inline dim3 grid_of(long long blocks) {
  if (blocks <= kGridX) return dim3((unsigned)blocks);
  return dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
// The block's number; past the last block behind the end of a second axis' last row.
__device__ inline size_t block_of_grid() { return blockIdx.y * (size_t)kGridX + blockIdx.x; }

}  // namespace qmoe
