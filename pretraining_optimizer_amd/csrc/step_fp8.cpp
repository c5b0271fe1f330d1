// Host side of muonh_step_quantized: the MuonH step whose update also writes the
// block-scaled FP8 forms of the updated weights.  The handle keeps a tile table
// (fixed by the shapes) and a table of output addresses (uploaded when they
// change), both made by the first such step.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <memory>
#include <string>
#include <vector>

#include "operators.h"
#include "step_tail.h"

using namespace muonh;

namespace {

int fail(int code, const std::string& msg) { return set_last_error(code, msg.c_str()); }

struct QuantizedStep {
  int64_t ntiles = 0;
  StepTile* d_tiles = nullptr;
  QuantArgs* d_outs = nullptr;
  QuantArgs* staging = nullptr;      // pinned
  std::vector<QuantArgs> current;    // what the device table holds
  hipEvent_t uploaded = nullptr;
  bool pending = false;

  ~QuantizedStep() {
    if (pending) (void)hipEventSynchronize(uploaded);
    if (uploaded) (void)hipEventDestroy(uploaded);
    if (d_tiles) (void)hipFree(d_tiles);
    if (d_outs) (void)hipFree(d_outs);
    if (staging) (void)hipHostFree(staging);
  }
};

#define QSTEP_HIP(expr)                                                                 \
  do {                                                                                  \
    hipError_t e_ = (expr);                                                             \
    if (e_ != hipSuccess)                                                               \
      return fail(MUONH_EHIP, std::string(#expr) + ": " + hipGetErrorString(e_));       \
  } while (0)

// The tables of a handle's first quantised step.
int make_tables(const muonh_matrix_desc* mats, int32_t n, std::shared_ptr<QuantizedStep>& out) {
  auto q = std::make_shared<QuantizedStep>();
  std::vector<StepTile> tiles;
  for (int32_t i = 0; i < n; ++i)
    for (int64_t r = 0; r * kFp8Tile < mats[i].rows; ++r)
      for (int64_t c = 0; c * kFp8Tile < mats[i].cols; ++c)
        tiles.push_back(StepTile{i, (uint32_t)r, (uint32_t)c});
  q->ntiles = (int64_t)tiles.size();
  if (hipMalloc(reinterpret_cast<void**>(&q->d_tiles), sizeof(StepTile) * tiles.size()) != hipSuccess ||
      hipMalloc(reinterpret_cast<void**>(&q->d_outs), sizeof(QuantArgs) * n) != hipSuccess ||
      hipHostMalloc(reinterpret_cast<void**>(&q->staging), sizeof(QuantArgs) * n, hipHostMallocDefault) != hipSuccess)
    return fail(MUONH_ENOMEM, "allocation of the quantised step's tables failed");
  QSTEP_HIP(hipEventCreateWithFlags(&q->uploaded, hipEventDisableTiming));
  QSTEP_HIP(hipMemcpy(q->d_tiles, tiles.data(), sizeof(StepTile) * tiles.size(), hipMemcpyHostToDevice));
  out = std::move(q);
  return MUONH_OK;
}

struct Context {
  muonh_handle* h;
  const muonh_matrix_desc* mats;
  int32_t n;
  const std::vector<QuantArgs>* outs;
  QuantizedStep* step;
};

int prepare(void* context, hipStream_t st) {
  auto* c = static_cast<Context*>(context);
  std::shared_ptr<void>& ext = step_extension(c->h);
  if (!ext) {
    std::shared_ptr<QuantizedStep> made;
    const int rc = make_tables(c->mats, c->n, made);
    if (rc) return rc;
    ext = made;
  }
  auto* q = static_cast<QuantizedStep*>(ext.get());
  c->step = q;
  const size_t bytes = sizeof(QuantArgs) * c->n;
  if (q->current.empty() || std::memcmp(q->current.data(), c->outs->data(), bytes) != 0) {
    // the staging copy is reused: the device must have read the previous upload
    if (q->pending) {
      QSTEP_HIP(hipEventSynchronize(q->uploaded));
      q->pending = false;
    }
    q->current.clear();   // unknown until the upload is enqueued
    std::memcpy(q->staging, c->outs->data(), bytes);
    QSTEP_HIP(hipMemcpyAsync(q->d_outs, q->staging, bytes, hipMemcpyHostToDevice, st));
    QSTEP_HIP(hipEventRecord(q->uploaded, st));
    q->pending = true;
    q->current = *c->outs;
  }
  return MUONH_OK;
}

hipError_t launch(void* context, int bf16, const MatGeom* geo, const MatPtrs* ptrs, const MatScalars* scal,
                  hipStream_t st) {
  const QuantizedStep* q = static_cast<Context*>(context)->step;
  return launch_update_quantize(bf16, q->d_tiles, q->ntiles, q->d_outs, geo, ptrs, scal, st);
}

// Form f of matrix i (rows x cols): nothing if its data is NULL.
int check_form(const muonh_fp8_matrix& f, const muonh_matrix_desc& d, int64_t rows, int64_t cols,
               const std::string& who) {
  if (f.rows != rows || f.cols != cols) return fail(MUONH_EINVAL, who + ": shape differs from the weight's");
  if (f.block_rows != 128) return fail(MUONH_EINVAL, who + ": block_rows must be 128");
  const int rc = check_fp8_matrix(f, who.c_str());
  if (rc) return rc;
  const int64_t count = d.rows * d.cols;
  if (fp8_overlaps(f, d.w, count * 4) || fp8_overlaps(f, d.m, count * 4) ||
      fp8_overlaps(f, d.g, count * (d.g_dtype == MUONH_BF16 ? 2 : 4)))
    return fail(MUONH_EINVAL, who + ": overlaps the weight, its gradient or its momentum");
  return MUONH_OK;
}

}  // namespace

extern "C" int muonh_step_quantized(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
                                    const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt,
                                    const muonh_step_args* args, void* stream) {
  return guarded([&]() -> int {
    if (!h || !args || !mats) return fail(MUONH_EINVAL, "null argument");
    if (n < 1) return fail(MUONH_EINVAL, "matrix count must be >= 1");
    if (!q && !qt) return fail(MUONH_EINVAL, "neither form is asked for");
    std::vector<QuantArgs> outs(n);
    for (int32_t i = 0; i < n; ++i) {
      const std::string name = "matrix " + std::to_string(i);
      QuantArgs& a = outs[i];
      std::memset(&a, 0, sizeof(a));
      a.rows = mats[i].rows;
      a.cols = mats[i].cols;
      int rc;
      if (q && q[i].data) {
        if ((rc = check_form(q[i], mats[i], a.rows, a.cols, name + " q"))) return rc;
        set_row_form(a, q[i]);
      }
      if (qt && qt[i].data) {
        if ((rc = check_form(qt[i], mats[i], a.cols, a.rows, name + " qt"))) return rc;
        set_column_form(a, qt[i]);
      }
    }
    // an output named twice would be written by two matrices at once
    std::vector<const void*> named;
    for (const QuantArgs& a : outs)
      for (const void* p : {(const void*)a.q, (const void*)a.qt, (const void*)a.s, (const void*)a.st})
        if (p) named.push_back(p);
    std::sort(named.begin(), named.end());
    if (std::adjacent_find(named.begin(), named.end()) != named.end())
      return fail(MUONH_EINVAL, "an output is named twice");
    Context c{h, mats, n, &outs, nullptr};
    return step_with_tail(h, mats, n, args, reinterpret_cast<hipStream_t>(stream),
                          StepTail{prepare, launch, &c});
  });
}
