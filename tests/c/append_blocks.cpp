// The blocks that an append touches, against 64-bit arithmetic, at sizes up to the largest a
// call takes (2^31 - 2^16 token rows, counts of new rows up to 2^31 - 1).
#include <cstdio>
#include <cstdlib>

#include "kv_blocks.h"

int main() {
  const int most = 0x7fff0000, any = 0x7fffffff;
  const int sizes[] = {1, 15, 16, 17, 127, 128, 129, 1000, 1 << 20, 1 << 30, most - 129, most - 1, most};
  const int counts[] = {0, 1, 2, 15, 16, 17, 128, 129, 100000, 1 << 30, most, any};
  const int blocks[] = {16, 32, 64, 128};
  long long checked = 0;
  for (const int blk : blocks)
    for (int S : sizes)
      for (int L : sizes)
        for (int T : counts)
          for (int n : counts) {
            if (L > S || n > L || n > T || T < 1) continue;
            const long long slots = gqa::append_slots(T, S, blk);
            const long long first = L - n, last = n ? (L - 1LL) / blk : -1, first_blk = first / blk;
            const long long touched = n ? last - first_blk + 1 : 0;
            if (slots < touched || slots > (long long)S / blk + 1 || slots > ((long long)T + blk - 2) / blk + 1) {
              std::printf("slots %lld of %lld: S %d L %d T %d n %d blk %d\n", slots, touched, S, L, T, n, blk);
              return 1;
            }
            const long long near[] = {0, 1, 2, touched - 2, touched - 1, touched, touched + 1, slots / 2, slots - 2, slots - 1};
            for (long long s : near) {
              if (s < 0 || s >= slots) continue;
              const long long want = s < touched ? (first_blk + s) * blk : -1;
              const int got = gqa::append_block_start(L, n, static_cast<int>(s), blk);
              ++checked;
              if (got != want) {
                std::printf("slot %lld: %d, not %lld: S %d L %d T %d n %d blk %d\n", s, got, want, S, L, T, n, blk);
                return 1;
              }
            }
          }
  std::printf("append_blocks: ok (%lld)\n", checked);
  return 0;
}
