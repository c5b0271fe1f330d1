// Prints how the FP8 product runs for sizes read from standard input, one per
// line: m n k block_a block_b c_bf16 -> ma nb splits split_blocks direct.
#include <cstdio>

#include "../../pretraining_optimizer_amd/csrc/operators.h"

using namespace muonh;

namespace muonh {
int set_last_error(int code, const char*) { return code; }
hipError_t launch_block_quantize(int, int, const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_block_matmul(int, const MatmulPlan&, const BlockMatmulArgs&, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_norm_forward(int, int, const NormArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm_backward(int, int, const NormGradArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t norm_partial_rows(int64_t rows, int64_t) { return rows; }
}  // namespace muonh

int main() {
  long long m, n, k;
  int ba, bb, bf16;
  while (std::scanf("%lld %lld %lld %d %d %d", &m, &n, &k, &ba, &bb, &bf16) == 6) {
    BlockMatmulArgs a{};
    a.m = (int32_t)m;
    a.n = (int32_t)n;
    a.kblocks = (int32_t)((k + 127) / 128);
    a.lda = a.ldb = (int64_t)a.kblocks * 128;
    a.ldsa = a.ldsb = (a.kblocks + 3) / 4 * 4;
    a.a_shift = ba == 128 ? 7 : 0;
    a.b_shift = bb == 128 ? 7 : 0;
    const MatmulPlan p = plan_block_matmul(bf16, a);
    std::printf("%d %d %d %d %d\n", p.ma, p.nb, p.splits, p.split_blocks, p.ma == 0 && narrow_direct(a) ? 1 : 0);
  }
  return 0;
}
