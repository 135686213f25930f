// Every unit and split of every head of an attention is taken by exactly one
// workgroup, whatever the number of heads, and chiplets share out the heads.
#include <cstdio>
#include <vector>

#include "ltc_cache.h"

int main() {
  long checked = 0;
  for (uint32_t heads = 1; heads <= 72; ++heads)
    for (uint32_t units : {1u, 2u, 3u, 7u, 8u, 33u, 101u})
      for (uint32_t splits : {1u, 2u, 3u, 5u, 64u}) {
        const uint32_t share = ltc::chiplet_share(heads), per_head = (units * splits + share - 1) / share * share;
        const uint32_t groups = per_head * heads;
        if (groups % 8) return std::printf("heads %u: %u workgroups\n", heads, groups), 1;
        std::vector<uint32_t> taken((size_t)heads * units * splits, 0), chiplets(heads, 0);
        // numbers past the last, as a grid of two dimensions has them, find no work
        for (uint32_t id = 0; id < groups + 64; ++id) {
          uint32_t head, unit, split;
          ltc::place(id, heads, splits, per_head, &head, &unit, &split);
          if (head >= heads || unit >= units) continue;
          if (id >= groups || split >= splits) return std::printf("heads %u id %u\n", heads, id), 1;
          ++taken[((size_t)head * units + unit) * splits + split];
          chiplets[head] |= 1u << id % 8;
          ++checked;
        }
        for (uint32_t n : taken)
          if (n != 1) return std::printf("heads %u units %u splits %u: taken %u times\n", heads, units, splits, n), 1;
        for (uint32_t c : chiplets)
          if ((uint32_t)__builtin_popcount(c) > share) return std::printf("heads %u: chiplets %x\n", heads, c), 1;
      }
  std::printf("%ld ok\n", checked);
}
