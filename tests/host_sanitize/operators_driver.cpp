// Drives the host code of the FP8 operators and the norms (operators.cpp,
// step_fp8.cpp) with no device: the product's plans over many sizes, refusals,
// and calls that have nothing to do.  Launchers are stubs that report no device.
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <string>

#include "../../pretraining_optimizer_amd/csrc/operators.h"
#include "../../pretraining_optimizer_amd/csrc/step_tail.h"

using namespace muonh;

static std::string g_error;

namespace muonh {
int set_last_error(int code, const char* msg) {
  g_error = msg;
  return code;
}
int step_with_tail(muonh_handle*, const muonh_matrix_desc*, int32_t, const muonh_step_args*, hipStream_t,
                   const StepTail&) {
  return set_last_error(MUONH_ESTATE, "stub");
}
std::shared_ptr<void>& step_extension(muonh_handle*) {
  static std::shared_ptr<void> none;
  return none;
}
hipError_t launch_block_quantize(int, int, const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_update_quantize(int, const StepTile*, int64_t, const QuantArgs*, const MatGeom*, const MatPtrs*,
                                  const MatScalars*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_block_matmul(int, const MatmulPlan&, const BlockMatmulArgs&, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_norm_forward(int, int, const NormArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm_backward(int, int, const NormGradArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t norm_partial_rows(int64_t rows, int64_t) { return rows < 256 ? rows : 256; }
}  // namespace muonh

#define CHECK(x)                                                             \
  do {                                                                       \
    if (!(x)) {                                                              \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, g_error.c_str());      \
      std::exit(1);                                                          \
    }                                                                        \
  } while (0)

static void plans() {
  const int64_t sizes[] = {1, 15, 16, 17, 33, 64, 65, 200, 256, 777, 1000, 2048, 4100, 8192, 12288, 100000};
  const int64_t lengths[] = {0, 1, 127, 128, 129, 1500, 2048, 8192, 16384, 100000};
  int seen[5][5] = {};
  int split = 0;
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int64_t k : lengths)
        for (int bf16 = 0; bf16 < 2; ++bf16) {
          BlockMatmulArgs a{};
          a.m = (int32_t)m;
          a.n = (int32_t)n;
          a.kblocks = (int32_t)((k + 127) / 128);
          a.lda = a.ldb = (int64_t)a.kblocks * 128;
          a.ldsa = a.ldsb = (a.kblocks + 3) / 4 * 4;
          const MatmulPlan p = plan_block_matmul(bf16, a);
          CHECK(p.ma >= 0 && p.ma <= 4 && p.nb >= 0 && p.nb <= 4 && (p.ma == 0) == (p.nb == 0));
          seen[p.ma][p.nb]++;
          CHECK(p.splits >= 1 && p.splits <= 16);
          // every block once: whole ranges, and a rest that is not empty
          CHECK((int64_t)p.splits * p.split_blocks >= a.kblocks);
          CHECK(p.splits == 1 || (int64_t)(p.splits - 1) * p.split_blocks < a.kblocks);
          CHECK(p.splits == 1 || p.split_blocks % 4 == 0);
          CHECK(p.workspace_bytes == (p.splits > 1 ? sizeof(float) * (size_t)p.splits * (size_t)(m * n) : 0));
          split += p.splits > 1;
          if (m <= 16 || n <= 16 || k == 0) CHECK(p.ma == 0 && p.splits == 1);
          if (p.ma == 0) CHECK(p.splits == 1);
          if (m >= 256 && n >= 2048 && k >= 8192) CHECK(p.ma > 0);
          // panels beyond the tile kernel's 32-bit offsets go to the narrow kernels
          a.ldb = (int64_t)1 << 23;
          CHECK(plan_block_matmul(bf16, a).ma == 0);
        }
  CHECK(split > 0 && seen[0][0] && seen[1][1] && seen[2][2] && seen[4][3] && seen[3][4] && seen[4][4]);
}

static void refusals() {
  char* base = reinterpret_cast<char*>((uintptr_t)1 << 40);
  auto mat = [&](int64_t rows, int64_t cols, int32_t br, char* data) {
    return muonh_fp8_matrix{data, data + ((uintptr_t)1 << 36), rows, cols, (cols + 127) / 128 * 128,
                            (cols + 511) / 512 * 4, br, 0};
  };
  muonh_fp8_matrix a = mat(300, 500, 1, base), b = mat(200, 500, 128, base + ((uintptr_t)1 << 38));
  char* c = base + ((uintptr_t)1 << 39);
  size_t need = 0;
  CHECK(muonh_block_matmul_workspace(&a, &b, MUONH_F32, &need) == MUONH_OK);
  CHECK(muonh_block_matmul(&a, &b, c, MUONH_F32, 200, 0, nullptr, 0, nullptr) == MUONH_EHIP);
  CHECK(muonh_block_matmul(&a, &b, c, MUONH_F32, 199, 0, nullptr, 0, nullptr) == MUONH_EINVAL);
  muonh_fp8_matrix la = mat(400, 9000, 1, base), lb = mat(700, 9000, 1, base + ((uintptr_t)1 << 38));
  CHECK(muonh_block_matmul_workspace(&la, &lb, MUONH_F32, &need) == MUONH_OK && need > 0);
  CHECK(muonh_block_matmul(&la, &lb, c, MUONH_F32, 700, 0, nullptr, 0, nullptr) == MUONH_ENOMEM);
  CHECK(muonh_block_matmul(&la, &lb, c, MUONH_F32, 700, 0, base, need - 1, nullptr) == MUONH_ENOMEM);
  CHECK(muonh_block_matmul(&la, &lb, c, MUONH_F32, 700, 0, base + 64, need, nullptr) == MUONH_EINVAL);
  CHECK(muonh_block_quantize(c, MUONH_BF16, 300, 500, 500, &a, nullptr, nullptr) == MUONH_EHIP);
  CHECK(muonh_block_quantize(c, MUONH_BF16, 300, 500, 499, &a, nullptr, nullptr) == MUONH_EINVAL);

  muonh_matrix_desc d{};
  d.w = c;
  d.g = c + 4096 * 300;
  d.m = c + 8192 * 300;
  d.rows = 300;
  d.cols = 500;
  muonh_step_args args{};
  muonh_handle* h = reinterpret_cast<muonh_handle*>(base);   // only passed on to the stub
  muonh_fp8_matrix q = mat(300, 500, 128, base), qt = mat(500, 300, 128, base + ((uintptr_t)1 << 38));
  CHECK(muonh_step_quantized(h, &d, 1, &q, &qt, &args, nullptr) == MUONH_ESTATE);
  CHECK(muonh_step_quantized(h, &d, 1, nullptr, nullptr, &args, nullptr) == MUONH_EINVAL);
  CHECK(muonh_step_quantized(h, &d, 0, &q, &qt, &args, nullptr) == MUONH_EINVAL);
  CHECK(muonh_step_quantized(h, &d, 1, &qt, nullptr, &args, nullptr) == MUONH_EINVAL);
  CHECK(muonh_step_quantized(h, &d, 1, &a, nullptr, &args, nullptr) == MUONH_EINVAL);   // block_rows 1
  muonh_fp8_matrix over = mat(300, 500, 128, c + 1024);
  CHECK(muonh_step_quantized(h, &d, 1, &over, nullptr, &args, nullptr) == MUONH_EINVAL);
  muonh_matrix_desc two[2] = {d, d};
  muonh_fp8_matrix same[2] = {q, q};
  CHECK(muonh_step_quantized(h, two, 2, same, nullptr, &args, nullptr) == MUONH_EINVAL);
  CHECK(g_error.find("twice") != std::string::npos);
  // the second matrix's output on the first's rows, weight, gradient or momentum
  two[1].w = c + ((uintptr_t)1 << 24);
  two[1].g = c + ((uintptr_t)2 << 24);
  two[1].m = c + ((uintptr_t)3 << 24);
  two[0].g = c + ((uintptr_t)4 << 24);
  two[0].m = c + ((uintptr_t)5 << 24);
  muonh_fp8_matrix apart[2] = {q, mat(300, 500, 128, base + ((uintptr_t)1 << 30))};
  CHECK(muonh_step_quantized(h, two, 2, apart, nullptr, &args, nullptr) == MUONH_ESTATE);
  for (char* at : {base + 512 * 299, c + 256, c + ((uintptr_t)4 << 24), c + ((uintptr_t)5 << 24),
                   c + ((uintptr_t)1 << 24) - 256}) {
    muonh_fp8_matrix bad[2] = {q, mat(300, 500, 128, at)};
    bad[1].scale = base + ((uintptr_t)1 << 31);
    CHECK(muonh_step_quantized(h, two, 2, bad, nullptr, &args, nullptr) == MUONH_EINVAL);
    CHECK(g_error.find("overlaps") != std::string::npos);
  }
  // forms side by side in rows of 1024 bytes, their scales in rows of 8
  muonh_fp8_matrix side[2] = {q, q};
  for (int i = 0; i < 2; ++i) {
    side[i].ld = 1024;
    side[i].ld_scale = 8;
    side[i].data = base + 512 * i;
    side[i].scale = base + ((uintptr_t)1 << 36) + 4 * i;
  }
  CHECK(muonh_step_quantized(h, two, 2, side, nullptr, &args, nullptr) == MUONH_ESTATE);
  side[1].data = base + 384;
  CHECK(muonh_step_quantized(h, two, 2, side, nullptr, &args, nullptr) == MUONH_EINVAL);
}

int main() {
  plans();
  refusals();
  std::printf("all checks passed\n");
  return 0;
}
