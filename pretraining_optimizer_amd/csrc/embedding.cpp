// Host side of the embedding: argument checks, the workspace's layout and the
// launches.  These entry points keep no state.

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "embedding.h"
#include "operator_checks.h"
#include "operators.h"

using namespace muonh;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 20;

int check_sizes(int64_t count, int64_t rows, int64_t cols) {
  int rc;
  if ((rc = check_size(count, 0, "count")) || (rc = check_size(rows, 0, "rows"))) return rc;
  if (cols < 1 || cols > kMaxCols) return fail(MUONH_EINVAL, "cols must be in [1, 2^20]");
  // of no launch are there more than 256 threads along x per token
  if (count > kMaxThreads / 256) return fail(MUONH_EINVAL, "count is too large for one launch");
  return MUONH_OK;
}

int check_kinds(int32_t token_bytes, float scale) {
  if (token_bytes != 4 && token_bytes != 8) return fail(MUONH_EINVAL, "token_bytes must be 4 or 8");
  if (!std::isfinite(scale)) return fail(MUONH_EINVAL, "scale must be finite");
  return MUONH_OK;
}

int64_t size_of(int32_t dtype) { return dtype == MUONH_BF16 ? 2 : 4; }

// The parts of the backward pass's workspace, each from a multiple of 256 bytes on.
struct Parts {
  int64_t keys, digits, partials;   // bytes; keys four times
  int64_t total() const { return 4 * keys + digits + partials; }
};
Parts parts_of(int64_t count, int64_t rows, int64_t cols) {
  auto whole = [](int64_t bytes) { return ceil_div(bytes, (int64_t)kAlign) * (int64_t)kAlign; };
  if (count == 0) return Parts{0, 0, 0};
  const SortPlan plan = plan_sort(count, rows);
  const int64_t runs = ceil_div(count, sum_run(count));
  return Parts{whole(count * 4), plan.blocks > 1 ? whole(plan.blocks * kSortDigits * 4) : 0,
               runs > 1 ? whole(runs * 2 * cols * 4) : 0};
}

}  // namespace

extern "C" {

int muonh_embedding_forward(const muonh_embedding_args* g, void* stream) {
  return guarded([&]() -> int {
    if (!g) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_dtype(g->table_dtype, "table")) || (rc = check_dtype(g->out_dtype, "out"))) return rc;
    if ((rc = check_sizes(g->count, g->rows, g->cols)) || (rc = check_kinds(g->token_bytes, g->scale))) return rc;
    if ((rc = check_pitch(g->ld_table, g->rows, g->cols, "ld_table")) || (rc = check_pitch(g->ld_out, g->count, g->cols, "ld_out")))
      return rc;
    if (g->count == 0) return MUONH_OK;
    if (!g->tokens || !g->out || (g->rows > 0 && !g->table)) return fail(MUONH_EINVAL, "null pointer: tokens, table or out");
    const int64_t ts = size_of(g->table_dtype), os = size_of(g->out_dtype);
    if (!aligned(g->tokens, (uintptr_t)g->token_bytes) || !aligned(g->table, (uintptr_t)ts) || !aligned(g->out, (uintptr_t)os))
      return fail(MUONH_EINVAL, "misaligned pointer");
    const Span tokens{g->tokens, g->count * g->token_bytes}, table{g->table, extent(g->rows, g->cols, g->ld_table, ts)};
    if (clash({Span{g->out, extent(g->count, g->cols, g->ld_out, os)}}, {tokens, table}))
      return fail(MUONH_EINVAL, "out overlaps tokens or table");
    EmbeddingArgs a{};
    a.tokens = g->tokens;
    a.table = g->table;
    a.out = g->out;
    a.count = g->count;
    a.rows = g->rows;
    a.cols = g->cols;
    a.ldt = g->ld_table;
    a.ldo = g->ld_out;
    a.wide = g->token_bytes == 8;
    a.scale = g->scale;
    forget_older_errors();
    return launched(launch_embedding_forward(g->table_dtype == MUONH_BF16, g->out_dtype == MUONH_BF16, a,
                                             reinterpret_cast<hipStream_t>(stream)),
                    "embedding_forward");
  });
}

int muonh_embedding_backward_workspace(int64_t count, int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_sizes(count, rows, cols))) return rc;
    *bytes = (size_t)parts_of(count, rows, cols).total();
    return MUONH_OK;
  });
}

int muonh_embedding_backward(const muonh_embedding_grad_args* g, void* stream) {
  return guarded([&]() -> int {
    if (!g) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_dtype(g->dout_dtype, "dout")) || (rc = check_dtype(g->table_dtype, "dtable"))) return rc;
    if ((rc = check_sizes(g->count, g->rows, g->cols)) || (rc = check_kinds(g->token_bytes, g->scale))) return rc;
    if (g->reserved != 0) return fail(MUONH_EINVAL, "reserved != 0");
    if (g->accumulate != 0 && g->accumulate != 1) return fail(MUONH_EINVAL, "accumulate must be 0 or 1");
    if ((rc = check_pitch(g->ld_table, g->rows, g->cols, "ld_table")) || (rc = check_pitch(g->ld_dout, g->count, g->cols, "ld_dout")))
      return rc;
    if (g->rows == 0 || (g->count == 0 && g->accumulate)) return MUONH_OK;
    if (!g->dtable || (g->count > 0 && (!g->tokens || !g->dout))) return fail(MUONH_EINVAL, "null pointer: tokens, dout or dtable");
    const int64_t ds = size_of(g->dout_dtype), ts = size_of(g->table_dtype);
    if (!aligned(g->tokens, (uintptr_t)g->token_bytes) || !aligned(g->dout, (uintptr_t)ds) || !aligned(g->dtable, (uintptr_t)ts))
      return fail(MUONH_EINVAL, "misaligned pointer");
    const Parts parts = parts_of(g->count, g->rows, g->cols);
    const int64_t need = parts.total();
    if (need > 0 && (!g->workspace || g->workspace_bytes < (size_t)need))
      return fail(MUONH_ENOMEM, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned(g->workspace, kAlign)) return fail(MUONH_EINVAL, "workspace must be 256-byte aligned");
    const Span tokens{g->tokens, g->count * g->token_bytes}, dout{g->dout, extent(g->count, g->cols, g->ld_dout, ds)};
    const Span dtable{g->dtable, extent(g->rows, g->cols, g->ld_table, ts)}, ws{g->workspace, need};
    if (clash({dtable, ws}, {tokens, dout})) return fail(MUONH_EINVAL, "dtable or the workspace overlaps an input or the other");
    EmbeddingGradArgs a{};
    a.tokens = g->tokens;
    a.dout = g->dout;
    a.dtable = g->dtable;
    a.count = g->count;
    a.rows = g->rows;
    a.cols = g->cols;
    a.ldd = g->ld_dout;
    a.ldt = g->ld_table;
    a.wide = g->token_bytes == 8;
    a.accumulate = g->accumulate;
    a.scale = g->scale;
    if (need > 0) {
      uint8_t* at = static_cast<uint8_t*>(g->workspace);
      for (int i = 0; i < 2; ++i) {
        a.keys[i] = reinterpret_cast<uint32_t*>(at + (2 * i) * parts.keys);
        a.places[i] = reinterpret_cast<uint32_t*>(at + (2 * i + 1) * parts.keys);
      }
      a.digits = reinterpret_cast<uint32_t*>(at + 4 * parts.keys);
      a.partials = reinterpret_cast<float*>(at + 4 * parts.keys + parts.digits);
    }
    forget_older_errors();
    return launched(launch_embedding_backward(g->dout_dtype == MUONH_BF16, g->table_dtype == MUONH_BF16, a,
                                              reinterpret_cast<hipStream_t>(stream)),
                    "embedding_backward");
  });
}

}  // extern "C"
