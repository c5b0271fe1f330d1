// Host side of the residual addition with RMS norm and FP8 output, and of its
// gradient: argument checks and the launches.  These entry points keep no state.

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "operator_checks.h"
#include "operators.h"

using namespace muonh;

namespace {

// An FP8 output shares no memory with `span`.
bool apart(const muonh_fp8_matrix* m, Span s) { return !m || s.bytes == 0 || !fp8_overlaps(*m, s.p, s.bytes); }

int check_form(const muonh_fp8_matrix* m, int64_t rows, int64_t cols, const char* whose) {
  if (!m) return MUONH_OK;
  int rc;
  if ((rc = check_fp8_matrix(*m, whose))) return rc;
  if (m->rows != rows || m->cols != cols) return fail(MUONH_EINVAL, std::string(whose) + ": shape differs");
  if (m->block_rows != 1) return fail(MUONH_EINVAL, std::string(whose) + ": block_rows must be 1");
  return MUONH_OK;
}

}  // namespace

extern "C" {

int muonh_add_norm_quantize(const muonh_add_norm_args* g, const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt,
                            void* stream) {
  return guarded([&]() -> int {
    int rc;
    if (!g) return fail(MUONH_EINVAL, "null argument");
    if (!q && !qt) return fail(MUONH_EINVAL, "neither form is asked for");
    if ((rc = check_dtype(g->dtype, "x"))) return rc;
    if (!(g->eps >= 0.0f) || !std::isfinite(g->eps)) return fail(MUONH_EINVAL, "eps must be >= 0 and finite");
    if ((rc = check_norm_size(g->rows, g->cols))) return rc;
    if ((rc = check_pitch(g->ldx, g->rows, g->cols, "ldx"))) return rc;
    if (!g->residual && g->h) return fail(MUONH_EINVAL, "h must be NULL without a residual");
    if (g->residual && ((rc = check_pitch(g->ld_residual, g->rows, g->cols, "ld_residual")) ||
                        (rc = check_pitch(g->ldh, g->rows, g->cols, "ldh"))))
      return rc;
    if ((rc = check_form(q, g->rows, g->cols, "q")) || (rc = check_form(qt, g->cols, g->rows, "qt"))) return rc;
    if (g->rows == 0) return MUONH_OK;
    if (!g->x || !g->weight || !g->rstd || (g->residual && !g->h))
      return fail(MUONH_EINVAL, "null pointer: x, weight, rstd or h");
    const int64_t size = g->dtype == MUONH_BF16 ? 2 : 4;
    for (const void* p : {g->x, g->residual, (const void*)g->h})
      if (!aligned(p, (uintptr_t)size)) return fail(MUONH_EINVAL, "misaligned pointer");
    if (!aligned(g->weight, 4) || !aligned(g->rstd, 4)) return fail(MUONH_EINVAL, "misaligned pointer");
    const Span x{g->x, extent(g->rows, g->cols, g->ldx, size)}, w = vec(g->weight, g->cols), rstd = vec(g->rstd, g->rows);
    Span r{nullptr, 0}, h{nullptr, 0};
    if (g->residual) {
      r = Span{g->residual, extent(g->rows, g->cols, g->ld_residual, size)};
      h = Span{g->h, extent(g->rows, g->cols, g->ldh, size)};
      if (!may_share(g->h, g->ldh, g->x, g->ldx, g->rows, g->cols, size) ||
          !may_share(g->h, g->ldh, g->residual, g->ld_residual, g->rows, g->cols, size))
        return fail(MUONH_EINVAL, "h overlaps x or residual");
    }
    if (clash({rstd, h}, {w}) || clash({rstd}, {x, r})) return fail(MUONH_EINVAL, "an output overlaps an input or another output");
    for (const muonh_fp8_matrix* m : {q, qt}) {
      for (const Span& s : {x, r, h, w, rstd})
        if (!apart(m, s)) return fail(MUONH_EINVAL, "an FP8 output overlaps an input or another output");
      if (m && overlap(m->scale, fp8_scale_bytes(*m), m->data, fp8_data_bytes(*m)))
        return fail(MUONH_EINVAL, "an FP8 output overlaps an input or another output");
    }
    if (q && qt && (!apart(q, Span{qt->data, fp8_data_bytes(*qt)}) || !apart(q, Span{qt->scale, fp8_scale_bytes(*qt)})))
      return fail(MUONH_EINVAL, "an FP8 output overlaps an input or another output");
    if (ceil_div(g->rows, kFp8Tile) * ceil_div(g->cols, kFp8Tile) * kQuantizeThreads > kMaxThreads)
      return fail(MUONH_EINVAL, "x is too large for one launch");
    AddNormArgs a{};
    a.x = g->x;
    a.residual = g->residual;
    a.weight = g->weight;
    a.h = g->h;
    a.rstd = g->rstd;
    a.rows = g->rows;
    a.cols = g->cols;
    a.ldx = g->ldx;
    a.ldr = g->ld_residual;
    a.ldh = g->ldh;
    a.eps = g->eps;
    QuantArgs out{};
    out.x = g->residual ? g->h : g->x;
    out.ldx = g->residual ? g->ldh : g->ldx;
    out.rows = g->rows;
    out.cols = g->cols;
    if (q) set_row_form(out, *q);
    if (qt) set_column_form(out, *qt);
    if (q && add_norm_rows_quantize(g->cols)) {
      a.q = out.q;
      a.s = out.s;
      a.ldq = out.ldq;
      a.lds = out.lds;
      out.q = out.s = nullptr;
    }
    const int bf16 = g->dtype == MUONH_BF16;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    forget_older_errors();
    hipError_t e = launch_add_norm_rows(bf16, a, st);
    if (e == hipSuccess && (out.q || out.qt)) e = launch_norm_quantize(bf16, out, g->weight, g->rstd, st);
    return launched(e, "add_norm_quantize");
  });
}

int muonh_add_norm_backward(const muonh_add_norm_grad_args* b, void* stream) {
  return guarded([&]() -> int {
    int rc;
    if (!b) return fail(MUONH_EINVAL, "null argument");
    const muonh_norm_grad_args* g = &b->g;
    if ((rc = check_dtype(g->dtype, "h"))) return rc;
    if (g->kind != MUONH_NORM_RMS) return fail(MUONH_EINVAL, "kind must be MUONH_NORM_RMS");
    if (g->reserved != 0) return fail(MUONH_EINVAL, "reserved != 0");
    if (g->accumulate != 0 && g->accumulate != 1) return fail(MUONH_EINVAL, "accumulate must be 0 or 1");
    if ((rc = check_norm_size(g->rows, g->cols))) return rc;
    if ((rc = check_pitch(g->ld_dy, g->rows, g->cols, "ld_dy")) || (rc = check_pitch(g->ldx, g->rows, g->cols, "ldx")) ||
        (rc = check_pitch(g->ld_dx, g->rows, g->cols, "ld_dx")) || (rc = check_pitch(b->ld_dh, g->rows, g->cols, "ld_dh")))
      return rc;
    if (g->mean || g->dbias) return fail(MUONH_EINVAL, "mean and dbias must be NULL");
    if (!g->weight || !g->dweight) return fail(MUONH_EINVAL, "null pointer: weight or dweight");
    const int64_t size = g->dtype == MUONH_BF16 ? 2 : 4;
    if (g->rows > 0) {
      if (!g->dy || !g->x || !g->dx || !g->rstd || !b->dh) return fail(MUONH_EINVAL, "null pointer: dy, dh, h, dx or rstd");
      for (const void* p : {g->dy, g->x, (const void*)g->dx, b->dh})
        if (!aligned(p, (uintptr_t)size)) return fail(MUONH_EINVAL, "misaligned pointer");
      if (!may_share(g->dx, g->ld_dx, g->dy, g->ld_dy, g->rows, g->cols, size) ||
          !may_share(g->dx, g->ld_dx, g->x, g->ldx, g->rows, g->cols, size) ||
          !may_share(g->dx, g->ld_dx, b->dh, b->ld_dh, g->rows, g->cols, size))
        return fail(MUONH_EINVAL, "dx overlaps dy, dh or h");
    }
    if (!aligned(g->weight, 4) || !aligned(g->rstd, 4) || !aligned(g->dweight, 4))
      return fail(MUONH_EINVAL, "misaligned pointer");
    size_t need = 0;
    if ((rc = muonh_norm_backward_workspace(g->rows, g->cols, &need))) return rc;
    if (need > 0 && (!g->workspace || g->workspace_bytes < need))
      return fail(MUONH_ENOMEM, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned(g->workspace, kAlign)) return fail(MUONH_EINVAL, "workspace must be 256-byte aligned");
    const Span dy{g->dy, extent(g->rows, g->cols, g->ld_dy, size)}, x{g->x, extent(g->rows, g->cols, g->ldx, size)};
    const Span dh{b->dh, extent(g->rows, g->cols, b->ld_dh, size)}, dx{g->dx, extent(g->rows, g->cols, g->ld_dx, size)};
    const Span ws{g->workspace, (int64_t)need}, dweight = vec(g->dweight, g->cols);
    if (clash({dx, dweight, ws}, {vec(g->weight, g->cols), vec(g->rstd, g->rows)}) || clash({dweight, ws}, {dy, x, dh}))
      return fail(MUONH_EINVAL, "an output or the workspace overlaps an input or another output");
    NormGradArgs a{};
    a.dy = g->dy;
    a.x = g->x;
    a.weight = g->weight;
    a.rstd = g->rstd;
    a.dx = g->dx;
    a.dweight = g->dweight;
    a.partials = static_cast<float*>(g->workspace);
    a.rows = g->rows;
    a.cols = g->cols;
    a.lddy = g->ld_dy;
    a.ldx = g->ldx;
    a.lddx = g->ld_dx;
    a.accumulate = g->accumulate;
    a.dh = b->dh;
    a.lddh = b->ld_dh;
    forget_older_errors();
    return launched(launch_add_norm_backward(g->dtype == MUONH_BF16, a, reinterpret_cast<hipStream_t>(stream)),
                    "add_norm_backward");
  });
}

}  // extern "C"
