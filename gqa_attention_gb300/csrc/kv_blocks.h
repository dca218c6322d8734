// kv_blocks.h -- which blocks of tokens an append touches.  Plain C++, no CUDA types.
#pragma once

#if defined(__CUDACC__)
#define GQA_HD __host__ __device__ __forceinline__
#else
#define GQA_HD inline
#endif

namespace gqa {

// Blocks of `blk` tokens that T new tokens of a cache of S_max can touch, wherever they start.
GQA_HD long long append_slots(int T, int S_max, int blk) {
  const long long by_rows = ((long long)T + blk - 2) / blk, by_cache = S_max / blk;
  return (by_rows < by_cache ? by_rows : by_cache) + 1;
}

// First token of the slot-th block that n new tokens ending at token L (n <= L) touch, or -1
// past the last one.  Blocks are compared before the product: a slot counts up to T / blk,
// whatever n is, and first_new + T need not fit in 32 bits.
GQA_HD int append_block_start(int L, int n, int slot, int blk) {
  if (n < 1) return -1;
  const int at = (L - n) / blk + slot;  // (both below 2^28)
  return at > (L - 1) / blk ? -1 : at * blk;
}

}  // namespace gqa
