// Launchers of the attention kernels (attention.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/muonh.h"

namespace muonh {

constexpr int kAttentionThreads = 256;
constexpr int kAttentionRows = 128;   // rows of a workgroup, where there are enough of them
constexpr int64_t kAttentionCus = 256;

struct AttentionArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;                  // read by the backward pass
  float* lse;                     // [heads][tokens]
  const int32_t* cu;              // [sequences + 1]
  int64_t ldq, ldk, ldv, ldo;     // elements between tokens
  int32_t tokens, sequences, heads, kv_heads, dim;
  int32_t blocks;                 // set by the launchers: attention_blocks() of the kernel's rows
  float scale;
  int32_t zero_rest;              // MUONH_ZERO_*: results whose rows that no sequence holds become zeros
};
struct AttentionGradArgs {
  AttentionArgs a;
  const uint16_t* dout;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  int64_t lddo, lddq, lddk, lddv;
  float* row_lse;                 // [heads][tokens]: -lse log2 e
  float* row_delta;               // [heads][tokens]: -delta
};
// Blocks of `rows` rows of any sequences in so many tokens, each sequence's last one cut.
inline int64_t attention_blocks(int64_t tokens, int64_t sequences, int64_t rows) { return tokens / rows + sequences; }

hipError_t launch_attention_forward(const AttentionArgs& a, hipStream_t st);
hipError_t launch_attention_backward(const AttentionGradArgs& g, hipStream_t st);

}  // namespace muonh
