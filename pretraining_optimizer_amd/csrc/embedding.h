// Launchers of the embedding kernels (embedding.hip) and the layout of the backward
// pass's workspace.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace muonh {

struct EmbeddingArgs {
  const void* tokens;     // int32 or int64
  const void* table;
  void* out;
  int64_t count, rows, cols, ldt, ldo;
  int32_t wide;           // tokens are int64
  float scale;
};
hipError_t launch_embedding_forward(int table_bf16, int out_bf16, const EmbeddingArgs& a, hipStream_t st);

constexpr int kSortThreads = 1024;
// Up to 8192 tokens, and up to 16384 whose keys would take several passes, are ranked
// among each other; of others, a workgroup sorts 4096.  Whole gradient into rows of 64
// columns, in us, ranked and sorted: 8192 tokens of 300 rows (a pass) 24 and 25.5, 16384 of them
// 38.0 and 24.7; of 151936 rows (two passes) 12288 tokens 35.1 and 41, 16384 40.4 and 41.4.
constexpr int kSortAlone = 16, kSortBeside = 4;             // per thread
constexpr int64_t kSortBlock = kSortThreads * kSortBeside;
constexpr int kSortDigits = 1024;                           // at most, of one pass
// Of up to so many workgroups each finds by itself where its keys of a digit begin, more
// have a launch for it.
constexpr int64_t kOwnBegin = 32;

// A token's key is its row, or `rows` if it has none.  Keys are sorted in passes of
// equally many bits, at most 10.
struct SortPlan {
  int32_t passes, bits;
  int64_t blocks;   // workgroups
};
inline SortPlan plan_sort(int64_t count, int64_t rows) {
  int bits = 1;
  while (((int64_t)1 << bits) <= rows) ++bits;
  const int passes = (bits + 9) / 10;
  const bool alone = count <= kSortThreads * (passes > 1 ? kSortAlone : kSortAlone / 2);
  return SortPlan{passes, (bits + passes - 1) / passes, alone ? 1 : (count + kSortBlock - 1) / kSortBlock};
}
// Sorted tokens that one group of threads adds up.
inline int64_t sum_run(int64_t count) { return count <= 65536 ? 16 : 64; }

struct EmbeddingGradArgs {
  const void* tokens;
  const void* dout;
  void* dtable;
  int64_t count, rows, cols, ldd, ldt;
  int32_t wide, accumulate;
  float scale;
  // workspace
  uint32_t* keys[2];      // [count], sorted in turn
  uint32_t* places[2];    // [count]: where each key's token stands
  uint32_t* digits;       // [blocks][kSortDigits]
  float* partials;        // [runs][2][cols]
};
hipError_t launch_embedding_backward(int dout_bf16, int table_bf16, const EmbeddingGradArgs& a, hipStream_t st);

}  // namespace muonh
