// Drives what muonh_step_quantized keeps between steps (its tables) with HIP itself
// as a stub: device memory is host memory, any call can be made to fail.  The step
// is a stub that, as the library's, runs the tail's check, its preparation and its
// launch.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <string>
#include <vector>

#include "../../pretraining_optimizer_amd/csrc/operators.h"
#include "../../pretraining_optimizer_amd/csrc/step_tail.h"

using namespace muonh;

// --- HIP ------------------------------------------------------------------
static int g_calls = 0, g_fail_at = -1;   // the call that fails, counted from 0
static hipError_t g_last = hipSuccess;
static int g_live = 0, g_uploads = 0, g_waits = 0;
static hipStreamCaptureStatus g_capture = hipStreamCaptureStatusNone;

static hipError_t call() {
  if (g_calls++ != g_fail_at) return hipSuccess;
  g_last = hipErrorOutOfMemory;
  return g_last;
}
static hipError_t take(void** p, size_t n) {
  const hipError_t e = call();
  if (e != hipSuccess) return e;
  *p = std::malloc(n);
  ++g_live;
  return hipSuccess;
}
static hipError_t give(void* p) {
  std::free(p);
  --g_live;
  return hipSuccess;
}
extern "C" {
hipError_t hipMalloc(void** p, size_t n) { return take(p, n); }
hipError_t hipFree(void* p) { return give(p); }
hipError_t hipHostMalloc(void** p, size_t n, unsigned int) { return take(p, n); }
hipError_t hipHostFree(void* p) { return give(p); }
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) { return take(reinterpret_cast<void**>(e), 8); }
hipError_t hipEventDestroy(hipEvent_t e) { return give(e); }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return call(); }
hipError_t hipEventSynchronize(hipEvent_t) {
  ++g_waits;
  return call();
}
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind) {
  const hipError_t e = call();
  if (e == hipSuccess) std::memcpy(d, s, n);
  return e;
}
hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, hipMemcpyKind, hipStream_t) {
  const hipError_t e = call();
  if (e == hipSuccess) {
    std::memcpy(d, s, n);
    ++g_uploads;
  }
  return e;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = g_capture;
  return hipSuccess;
}
hipError_t hipGetLastError(void) {
  const hipError_t e = g_last;
  g_last = hipSuccess;
  return e;
}
const char* hipGetErrorString(hipError_t) { return "stub error"; }
}

// --- the library ------------------------------------------------------------
static std::string g_error;
static std::shared_ptr<void> g_extension;
static std::vector<QuantArgs> g_launched;   // the outputs that the last launch read
static int64_t g_tiles = 0;
static int32_t g_count = 0;

namespace muonh {
int set_last_error(int code, const char* msg) {
  g_error = msg;
  return code;
}
int step_with_tail(muonh_handle*, const muonh_matrix_desc*, int32_t n, const muonh_step_args*, hipStream_t st,
                   const StepTail& tail) {
  g_count = n;
  int rc = tail.check(tail.context, nullptr, 0);
  if (rc) return rc;
  if ((rc = tail.prepare(tail.context, st))) return rc;
  return tail.launch(tail.context, 1, nullptr, nullptr, nullptr, st) == hipSuccess ? MUONH_OK : MUONH_EHIP;
}
std::shared_ptr<void>& step_extension(muonh_handle*) { return g_extension; }
hipError_t launch_update_quantize(int, const StepTile* tiles, int64_t ntiles, const QuantArgs* outs, const MatGeom*,
                                  const MatPtrs*, const MatScalars*, hipStream_t) {
  g_launched.assign(outs, outs + g_count);
  g_tiles = ntiles;
  for (int64_t i = 0; i < ntiles; ++i)   // every tile inside its matrix
    if (tiles[i].mat < 0 || tiles[i].mat >= g_count || (int64_t)tiles[i].tr * kFp8Tile >= outs[tiles[i].mat].rows ||
        (int64_t)tiles[i].tc * kFp8Tile >= outs[tiles[i].mat].cols)
      return hipErrorInvalidValue;
  return hipSuccess;
}
hipError_t launch_block_quantize(int, int, const QuantArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_block_matmul(int, const MatmulPlan&, const BlockMatmulArgs&, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_forward(int, int, const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_backward(int, int, const NormGradArgs&, hipStream_t) { return hipSuccess; }
int64_t norm_partial_rows(int64_t rows, int64_t) { return rows; }
}  // namespace muonh

#define CHECK(x)                                                        \
  do {                                                                  \
    if (!(x)) {                                                         \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, g_error.c_str()); \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

static char* const kBase = reinterpret_cast<char*>((uintptr_t)1 << 40);
static muonh_handle* const kHandle = reinterpret_cast<muonh_handle*>(kBase);   // only passed on to the stub

int main() {
  // 300 x 500 and 129 x 128: 3 x 4 and 2 x 1 tiles
  muonh_matrix_desc d[2]{};
  for (int i = 0; i < 2; ++i) {
    d[i].w = kBase + ((uintptr_t)(1 + 3 * i) << 24);
    d[i].g = kBase + ((uintptr_t)(2 + 3 * i) << 24);
    d[i].m = kBase + ((uintptr_t)(3 + 3 * i) << 24);
  }
  d[0].rows = 300, d[0].cols = 500, d[1].rows = 129, d[1].cols = 128;
  muonh_step_args args{};
  auto step = [&](int shift) {
    char* at = kBase + ((uintptr_t)1 << 32) + ((uintptr_t)shift << 28);
    muonh_fp8_matrix q[2] = {{at, at + (1 << 24), 300, 500, 512, 4, 128, 0},
                             {at + (2 << 24), at + (3 << 24), 129, 128, 128, 4, 128, 0}};
    return muonh_step_quantized(kHandle, d, 2, q, nullptr, &args, nullptr);
  };
  // the calls of a first step; every one of them failing in turn leaves nothing
  // allocated that is not kept, no pending error, and a handle that still works
  CHECK(step(0) == MUONH_OK && g_tiles == 14 && g_uploads == 1 && g_waits == 0);
  const int first = g_calls;
  CHECK(first >= 6);
  g_extension.reset();
  CHECK(g_live == 0);
  for (int k = 0; k < first; ++k) {
    g_calls = 0, g_fail_at = k;
    const int rc = step(0);
    CHECK(rc == MUONH_ENOMEM || rc == MUONH_EHIP);
    CHECK(hipGetLastError() == hipSuccess);
    g_fail_at = -1;
    CHECK(step(1) == MUONH_OK);
    CHECK(g_launched.size() == 2 && g_launched[0].q == (uint8_t*)kBase + ((uintptr_t)1 << 32) + ((uintptr_t)1 << 28));
    CHECK(step(0) == MUONH_OK);
    CHECK(g_launched[0].q == (uint8_t*)kBase + ((uintptr_t)1 << 32) && g_launched[1].qt == nullptr);
    g_extension.reset();
    CHECK(g_live == 0);
  }
  // the same outputs again are not uploaded; others wait for the previous upload
  g_uploads = g_waits = 0;
  for (int k = 0; k < 3; ++k) CHECK(step(0) == MUONH_OK);
  CHECK(g_uploads == 1 && g_waits == 0);
  CHECK(step(1) == MUONH_OK && g_uploads == 2 && g_waits == 1);
  CHECK(step(0) == MUONH_OK && g_uploads == 3 && g_waits == 2);
  // an upload that fails is made again, with the same outputs too
  for (int k = 0; k < 3; ++k) {
    g_calls = 0, g_fail_at = k;
    CHECK(step(1) == MUONH_EHIP && hipGetLastError() == hipSuccess);
    g_fail_at = -1;
    CHECK(step(1) == MUONH_OK);
    CHECK(g_launched[0].q == (uint8_t*)kBase + ((uintptr_t)1 << 32) + ((uintptr_t)1 << 28));
    CHECK(step(0) == MUONH_OK && g_launched[0].q == (uint8_t*)kBase + ((uintptr_t)1 << 32));
  }
  // a stream that is being captured: nothing is called
  g_capture = hipStreamCaptureStatusActive;
  g_calls = 0;
  CHECK(step(1) == MUONH_ESTATE && g_calls == 0);
  g_capture = hipStreamCaptureStatusNone;
  g_extension.reset();
  CHECK(g_live == 0);
  std::printf("all checks passed\n");
  return 0;
}
