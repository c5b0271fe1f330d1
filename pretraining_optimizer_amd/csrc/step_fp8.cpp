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
    if (e_ != hipSuccess) {                                                             \
      forget_older_errors(); /* reported here */                                        \
      return fail(MUONH_EHIP, std::string(#expr) + ": " + hipGetErrorString(e_));       \
    }                                                                                   \
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
      hipHostMalloc(reinterpret_cast<void**>(&q->staging), sizeof(QuantArgs) * n, hipHostMallocDefault) != hipSuccess) {
    forget_older_errors();
    return fail(MUONH_ENOMEM, "allocation of the quantised step's tables failed");
  }
  QSTEP_HIP(hipEventCreateWithFlags(&q->uploaded, hipEventDisableTiming));
  QSTEP_HIP(hipMemcpy(q->d_tiles, tiles.data(), sizeof(StepTile) * tiles.size(), hipMemcpyHostToDevice));
  out = std::move(q);
  return MUONH_OK;
}

struct Context {
  muonh_handle* h;
  const muonh_matrix_desc* mats;
  int32_t n;
  const muonh_fp8_matrix* q;
  const muonh_fp8_matrix* qt;
  const std::vector<QuantArgs>* outs;
  QuantizedStep* step;
};

// No output lies in the handle's workspace, from which the launches read the
// update, the coefficients and their tables while others write the outputs.
int check(void* context, const void* workspace, size_t bytes) {
  const auto* c = static_cast<const Context*>(context);
  for (int32_t i = 0; i < c->n; ++i)
    for (const muonh_fp8_matrix* f : {c->q, c->qt})
      if (f && f[i].data && fp8_overlaps(f[i], workspace, (int64_t)bytes))
        return fail(MUONH_EINVAL, "matrix " + std::to_string(i) + ": an output overlaps the handle's workspace");
  return MUONH_OK;
}

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

// The form f of a weight, rows x cols.
int check_form(const muonh_fp8_matrix& f, int64_t rows, int64_t cols, const std::string& who) {
  if (f.rows != rows || f.cols != cols) return fail(MUONH_EINVAL, who + ": shape differs from the weight's");
  if (f.block_rows != 128) return fail(MUONH_EINVAL, who + ": block_rows must be 128");
  return check_fp8_matrix(f, who.c_str());
}

// Memory of a step: rows of `width` bytes, `pitch` bytes apart.
struct Span {
  uintptr_t begin, end;
  int64_t width, pitch;
  bool out;
};
// Sizes that are out of range belong to no handle's matrices: such a step is
// refused by its own checks.
bool in_range(int64_t v) { return v >= 1 && v <= (int64_t)1 << 30; }

// Whether an output shares memory with another, or with a weight, gradient or
// momentum: two workgroups would write it, or one read what another writes.
// Forms side by side in rows of one pitch do not.
bool outputs_overlap(const muonh_matrix_desc* mats, int32_t n, const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt) {
  std::vector<Span> spans;
  auto add = [&](const void* p, int64_t bytes, int64_t width, int64_t pitch, bool out) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p && bytes > 0) spans.push_back(Span{at, at + (uintptr_t)bytes, width, pitch, out});
  };
  for (int32_t i = 0; i < n; ++i) {
    if (in_range(mats[i].rows) && in_range(mats[i].cols)) {
      const int64_t count = mats[i].rows * mats[i].cols;
      const int64_t g_bytes = count * (mats[i].g_dtype == MUONH_BF16 ? 2 : 4);
      add(mats[i].w, count * 4, count * 4, count * 4, false);
      add(mats[i].m, count * 4, count * 4, count * 4, false);
      add(mats[i].g, g_bytes, g_bytes, g_bytes, false);
    }
    for (const muonh_fp8_matrix* f : {q, qt})
      if (f && f[i].data) {
        add(f[i].data, fp8_data_bytes(f[i]), fp8_data_width(f[i]), f[i].ld, true);
        add(f[i].scale, fp8_scale_bytes(f[i]), fp8_scale_width(f[i]), f[i].ld_scale, true);
      }
  }
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.begin < y.begin; });
  for (size_t i = 0; i < spans.size(); ++i)
    for (size_t j = i + 1; j < spans.size() && spans[j].begin < spans[i].end; ++j) {
      const Span &x = spans[i], &y = spans[j];
      if (!x.out && !y.out) continue;
      const int64_t d = (int64_t)(y.begin - x.begin) % x.pitch;
      if (x.pitch != y.pitch || d < x.width || x.pitch - d < y.width) return true;
    }
  return false;
}

}  // namespace

extern "C" int muonh_step_quantized(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
                                    const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt,
                                    const muonh_step_args* args, void* stream) {
  return guarded([&]() -> int {
    if (!h || !args || !mats) return fail(MUONH_EINVAL, "null argument");
    if (n < 1) return fail(MUONH_EINVAL, "matrix count must be >= 1");
    if (!q && !qt) return fail(MUONH_EINVAL, "neither form is asked for");
    // the tables are allocated and uploaded from the host: not for a recording
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(reinterpret_cast<hipStream_t>(stream), &capture) == hipSuccess &&
        capture != hipStreamCaptureStatusNone)
      return fail(MUONH_ESTATE, "the stream is being captured");
    std::vector<QuantArgs> outs(n);
    for (int32_t i = 0; i < n; ++i) {
      const std::string name = "matrix " + std::to_string(i);
      QuantArgs& a = outs[i];
      std::memset(&a, 0, sizeof(a));
      a.rows = mats[i].rows;
      a.cols = mats[i].cols;
      int rc;
      if (q && q[i].data) {
        if ((rc = check_form(q[i], a.rows, a.cols, name + " q"))) return rc;
        set_row_form(a, q[i]);
      }
      if (qt && qt[i].data) {
        if ((rc = check_form(qt[i], a.cols, a.rows, name + " qt"))) return rc;
        set_column_form(a, qt[i]);
      }
    }
    if (outputs_overlap(mats, n, q, qt))
      return fail(MUONH_EINVAL, "an output is named twice, or overlaps another, a weight, a gradient or a momentum");
    Context c{h, mats, n, q, qt, &outs, nullptr};
    return step_with_tail(h, mats, n, args, reinterpret_cast<hipStream_t>(stream),
                          StepTail{check, prepare, launch, &c});
  });
}
