// decode_cut.cuh -- the cut of a decode batch by its sequences' lengths, which every CTA
// works out for itself.
#pragma once

#include "common.cuh"

namespace gqa {
namespace {

// A CTA's share of a batch whose splits follow the sequences' lengths: piece `split` of
// `count` of sequence b, each of `tiles` tiles (b < 0: none).
struct Piece {
  int b, split, count, tiles;
};
// The batch is cut into pieces of as many tiles as are needed for at most `pieces` of them
// (and n_split of a sequence; every sequence has one, also one of a bad length), and
// this CTA takes piece `index` in the order of the sequences.  One warp, lane i with
// the tiles of sequences i, 32 + i and 64 + i (0: a bad length); every warp of the
// grid finds the same cut.
constexpr int kMaxCut = 96;  // sequences
__device__ __noinline__ Piece find_piece(int t0, int t1, int t2, int B, int n_split, int pieces,
                                         int index, int lane) {
  const int total = t0 + t1 + t2;  // (each at most 2^25: 2^31 tokens in tiles of 64)
  const long long all = static_cast<long long>(__reduce_add_sync(0xffffffffu, total >> 12)) * 4096 +
                        __reduce_add_sync(0xffffffffu, total & 4095);
  const int most = max(1, __reduce_max_sync(0xffffffffu, max(max(t0, t1), t2)));
  auto cuts = [&](int t, int k, int c) {  // pieces of sequence 32 k + lane
    return 32 * k + lane < B ? max(1, (t + c - 1) / c) : 0;
  };
  int lo = max(1, static_cast<int>(max((all + pieces - 1) / pieces,
                                       (most + n_split - 1LL) / n_split)));
  // sum of ceil(t / c) <= all / c + B
  int hi = static_cast<int>(min((long long)most, max((long long)lo, all / (pieces - B) + 1)));
  while (lo < hi) {
    const int c = (lo + hi) / 2;
    const int need = cuts(t0, 0, c) + cuts(t1, 1, c) + cuts(t2, 2, c);
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, need)) <= pieces) hi = c;
    else lo = c + 1;
  }
  int left = index;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int mine = cuts(k == 0 ? t0 : k == 1 ? t1 : t2, k, hi);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, upto > left);
    if (past != 0) {
      const int who = __ffs(past) - 1;
      const int count = __shfl_sync(0xffffffffu, mine, who);
      return {32 * k + who, left - (__shfl_sync(0xffffffffu, upto, who) - count), count, hi};
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return {-1, 0, 0, hi};
}

}  // namespace
}  // namespace gqa
