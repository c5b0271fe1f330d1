// Drives muonh_step_quantized with no device: an output that shares memory with
// the handle's workspace is refused before anything is enqueued.  The step itself
// is a stub that, as the library's, asks the tail's check first.
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <string>

#include "../../pretraining_optimizer_amd/csrc/operators.h"
#include "../../pretraining_optimizer_amd/csrc/step_tail.h"

using namespace muonh;

static std::string g_error;
static char* const kBase = reinterpret_cast<char*>((uintptr_t)1 << 40);
static char* const kWorkspace = kBase + ((uintptr_t)1 << 34);
static const size_t kWorkspaceBytes = (size_t)1 << 20;
static int g_prepared = 0;

namespace muonh {
int set_last_error(int code, const char* msg) {
  g_error = msg;
  return code;
}
int step_with_tail(muonh_handle*, const muonh_matrix_desc*, int32_t, const muonh_step_args*, hipStream_t,
                   const StepTail& tail) {
  const int rc = tail.check(tail.context, kWorkspace, kWorkspaceBytes);
  if (rc) return rc;
  ++g_prepared;
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
int64_t norm_partial_rows(int64_t rows, int64_t) { return rows; }
}  // namespace muonh

#define CHECK(x)                                                        \
  do {                                                                  \
    if (!(x)) {                                                         \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, g_error.c_str()); \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

int main() {
  // 300 x 500: 300 rows of 512 bytes, 3 x 4 scales; 500 rows of 384, 4 x 4
  muonh_matrix_desc d[2]{};
  for (int i = 0; i < 2; ++i) {
    d[i].w = kBase + ((uintptr_t)(1 + 3 * i) << 24);
    d[i].g = kBase + ((uintptr_t)(2 + 3 * i) << 24);
    d[i].m = kBase + ((uintptr_t)(3 + 3 * i) << 24);
    d[i].rows = 300;
    d[i].cols = 500;
  }
  muonh_step_args args{};
  muonh_handle* h = reinterpret_cast<muonh_handle*>(kBase);   // only passed on to the stub
  auto form = [&](bool t, char* data, char* scale) {
    return t ? muonh_fp8_matrix{data, scale, 500, 300, 384, 4, 128, 0}
             : muonh_fp8_matrix{data, scale, 300, 500, 512, 4, 128, 0};
  };
  char* free_at = kBase + ((uintptr_t)1 << 32);
  auto step = [&](char* data, char* scale, bool t, int which) {
    muonh_fp8_matrix q[2], qt[2];
    for (int i = 0; i < 2; ++i) {
      q[i] = form(false, free_at + ((uintptr_t)i << 24), free_at + ((uintptr_t)(4 + i) << 24));
      qt[i] = form(true, free_at + ((uintptr_t)(8 + i) << 24), free_at + ((uintptr_t)(12 + i) << 24));
    }
    muonh_fp8_matrix& m = (t ? qt : q)[which];
    if (data) m.data = data;
    if (scale) m.scale = scale;
    return muonh_step_quantized(h, d, 2, q, qt, &args, nullptr);
  };
  char* const end = kWorkspace + kWorkspaceBytes;
  for (bool t : {false, true})
    for (int which = 0; which < 2; ++which) {
      const int64_t bytes = t ? 499 * 384 + 384 : 299 * 512 + 512;   // 384: three blocks
      const int64_t scales = t ? 3 * 4 + 4 : 2 * 4 + 4;
      for (char* at : {kWorkspace, kWorkspace - bytes + 16, kWorkspace + 4096, end - 16}) {
        CHECK(step(at, nullptr, t, which) == MUONH_EINVAL);
        CHECK(g_error.find("workspace") != std::string::npos);
      }
      for (char* at : {kWorkspace, kWorkspace - scales + 4, end - 4}) {
        CHECK(step(nullptr, at, t, which) == MUONH_EINVAL);
        CHECK(g_error.find("workspace") != std::string::npos);
      }
      CHECK(g_prepared == 0);
      // right before it and right behind it
      for (char* at : {kWorkspace - bytes, end}) CHECK(step(at, nullptr, t, which) == MUONH_ESTATE);
      for (char* at : {kWorkspace - scales, end}) CHECK(step(nullptr, at, t, which) == MUONH_ESTATE);
      CHECK(g_prepared == 4);
      g_prepared = 0;
    }
  // an entry that is not written may name anything
  muonh_fp8_matrix none[2] = {form(false, free_at, free_at + (1 << 24)), form(false, nullptr, kWorkspace)};
  CHECK(muonh_step_quantized(h, d, 2, none, nullptr, &args, nullptr) == MUONH_ESTATE);
  std::printf("all checks passed\n");
  return 0;
}
