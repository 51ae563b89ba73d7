// Which blocks' parts the join of a split segment takes (host and device; no CUDA types).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define KVQ_HD __host__ __device__ __forceinline__
#else
#define KVQ_HD inline
#endif

namespace kvq {

// What a block did with the segment it shares with the block before it. A block whose wait ran out may leave any of
// them, kSegBegins above all: it ends before it has handed its part on.
enum { kSegBegins = 0, kSegGoesOn = 1, kSegEnds = 2, kSegNoWork = 3 };

struct JoinParts {
  uint32_t parts;  // of the 32 blocks, those whose parts belong to the segment
  int state;       // 0: it goes on in the next 32, 1: complete, 2: cut off, nothing is to be read behind `parts`
};
// goes_on, ends: bit i of 32 blocks in order, the first of them behind the segment's so far. Blocks that do not exist
// have neither bit, so none of them is ever among the parts.
KVQ_HD JoinParts join_parts(uint32_t goes_on, uint32_t ends) {
  const uint32_t stop = ~goes_on;  // the segment passes every block below the lowest of these
  if (stop == 0) return {goes_on, 0};
  const uint32_t bit = stop & (0u - stop), below = bit - 1;
  if (ends & bit) return {below | bit, 1};
  return {below, 2};
}

}  // namespace kvq
