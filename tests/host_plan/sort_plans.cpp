// Prints how the embedding gradient orders its tokens for sizes read from standard input,
// one per line: tokens rows -> passes workgroups path.
#include <cstdio>

#include "../../pretraining_optimizer_amd/csrc/embedding.h"

using namespace muonh;

int main() {
  long long count, rows;
  while (std::scanf("%lld %lld", &count, &rows) == 2) {
    const SortPlan p = plan_sort(count, rows);
    std::printf("%d %lld %s\n", p.passes, (long long)p.blocks,
                p.blocks == 1 ? "ranked" : p.blocks <= kOwnBegin ? "own" : "begin");
  }
  return 0;
}
