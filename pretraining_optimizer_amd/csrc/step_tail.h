// A MuonH step with another last launch than the update, and what such a
// variant keeps with its handle.
#pragma once

#include <memory>

#include "internal.h"

namespace muonh {

// A step whose last launch is another than launch_update: `check` runs before
// anything is enqueued, with the handle's workspace (the caller's, where the
// options gave one); `prepare` after the step's own checks and uploads, before its
// first launch; `launch` in place of the update.  `context` is the caller's.
struct StepTail {
  int (*check)(void* context, const void* workspace, size_t bytes);
  int (*prepare)(void* context, hipStream_t st);
  hipError_t (*launch)(void* context, int bf16, const MatGeom* geo, const MatPtrs* ptrs,
                       const MatScalars* scal, hipStream_t st);
  void* context;
};
int step_with_tail(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
                   const muonh_step_args* args, hipStream_t st, const StepTail& tail);
// What such a variant keeps with the handle; released by muonh_destroy, after
// the handle's last stream has passed its work.
std::shared_ptr<void>& step_extension(muonh_handle* h);

}  // namespace muonh
