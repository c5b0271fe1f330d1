// Host side of the block-scaled FP8 operators and of the norms: argument
// checks, workspace sizes and the launches.  These entry points keep no state:
// everything a call needs beyond its arguments is in the caller's workspace.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "operator_checks.h"
#include "operators.h"

using namespace muonh;

// What a row of an operand takes: the quantiser writes zeros behind the columns.
int64_t muonh::fp8_data_width(const muonh_fp8_matrix& m) { return ceil_div(m.cols, kFp8Block) * kFp8Block; }
int64_t muonh::fp8_scale_width(const muonh_fp8_matrix& m) { return ceil_div(ceil_div(m.cols, kFp8Block), 4) * 4; }
int64_t muonh::fp8_data_bytes(const muonh_fp8_matrix& m) {
  return m.rows > 0 && m.cols > 0 ? extent(m.rows, fp8_data_width(m), m.ld, 1) : 0;
}
int64_t muonh::fp8_scale_bytes(const muonh_fp8_matrix& m) {
  return m.rows > 0 && m.cols > 0 ? extent(ceil_div(m.rows, m.block_rows), fp8_scale_width(m), m.ld_scale, 1) : 0;
}

int muonh::check_fp8_matrix(const muonh_fp8_matrix& m, const char* whose) {
  const std::string who = std::string(whose) + ": ";
  int rc;
  if ((rc = check_size(m.rows, 0, (who + "rows").c_str()))) return rc;
  if ((rc = check_size(m.cols, 0, (who + "cols").c_str()))) return rc;
  if (m.block_rows != 1 && m.block_rows != 128) return fail(MUONH_EINVAL, who + "block_rows must be 1 or 128");
  if (m.reserved != 0) return fail(MUONH_EINVAL, who + "reserved != 0");
  if ((rc = check_pitch(m.ld, m.rows, m.cols, (who + "ld").c_str()))) return rc;
  if (m.ld % kFp8Block != 0) return fail(MUONH_EINVAL, who + "ld must be a multiple of 128");
  if ((rc = check_pitch(m.ld_scale, m.rows, ceil_div(m.cols, kFp8Block), (who + "ld_scale").c_str()))) return rc;
  if (m.ld_scale % 4 != 0) return fail(MUONH_EINVAL, who + "ld_scale must be a multiple of 4");
  if (m.rows > 0 && m.cols > 0) {
    if (!m.data || !m.scale) return fail(MUONH_EINVAL, who + "null pointer");
    if (!aligned(m.data, 16) || !aligned(m.scale, 4))
      return fail(MUONH_EINVAL, who + "data must be 16-byte and scale 4-byte aligned");
  }
  return MUONH_OK;
}

void muonh::set_row_form(QuantArgs& a, const muonh_fp8_matrix& m) {
  a.q = static_cast<uint8_t*>(m.data);
  a.s = static_cast<uint8_t*>(m.scale);
  a.ldq = m.ld;
  a.lds = m.ld_scale;
}

void muonh::set_column_form(QuantArgs& a, const muonh_fp8_matrix& m) {
  a.qt = static_cast<uint8_t*>(m.data);
  a.st = static_cast<uint8_t*>(m.scale);
  a.ldqt = m.ld;
  a.ldst = m.ld_scale;
}

bool muonh::fp8_overlaps(const muonh_fp8_matrix& m, const void* p, int64_t bytes) {
  return overlap(m.data, fp8_data_bytes(m), p, bytes) || overlap(m.scale, fp8_scale_bytes(m), p, bytes);
}

namespace {

int check_operands(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b) {
  if (!a || !b) return fail(MUONH_EINVAL, "null operand");
  int rc;
  if ((rc = check_fp8_matrix(*a, "a"))) return rc;
  if ((rc = check_fp8_matrix(*b, "b"))) return rc;
  if (a->cols != b->cols) return fail(MUONH_EINVAL, "a.cols differs from b.cols");
  return MUONH_OK;
}

BlockMatmulArgs matmul_args(const muonh_fp8_matrix& a, const muonh_fp8_matrix& b) {
  BlockMatmulArgs p{};
  p.a = static_cast<const uint8_t*>(a.data);
  p.b = static_cast<const uint8_t*>(b.data);
  p.sa = static_cast<const uint8_t*>(a.scale);
  p.sb = static_cast<const uint8_t*>(b.scale);
  p.lda = a.ld;
  p.ldb = b.ld;
  p.ldsa = a.ld_scale;
  p.ldsb = b.ld_scale;
  p.m = (int32_t)a.rows;
  p.n = (int32_t)b.rows;
  p.kblocks = (int32_t)ceil_div(a.cols, kFp8Block);
  p.a_shift = a.block_rows == 128 ? 7 : 0;
  p.b_shift = b.block_rows == 128 ? 7 : 0;
  return p;
}

int check_vectors(bool ok, const char* what) {
  return ok ? MUONH_OK : fail(MUONH_EINVAL, std::string("null pointer: ") + what);
}

}  // namespace

namespace {

// Measured times of the tile kernel on an MI355X, in us: one block of 128 of the
// contraction with `per` workgroups on each CU (index per - 1), and what a round
// costs besides its blocks.  [0]: FP8 arithmetic (bf16 results), [1]: bf16
// arithmetic (fp32 results).
struct TileRate {
  int32_t ma, nb, per_cu;
  double block[2][4], round[2];
  // the least time of a block where operands beyond an XCD's L2 (kColdBytes) are
  // read by up to four tiles each, so from further away
  double cold[4];
};
constexpr int64_t kColdBytes = (int64_t)4 << 20;
constexpr TileRate kTileRates[] = {
    {4, 4, 1, {{1.61, 0, 0, 0}, {2.88, 0, 0, 0}}, {8.8, 16.3}, {1.7, 0, 0, 0}},
    {4, 3, 1, {{1.20, 0, 0, 0}, {2.17, 0, 0, 0}}, {10.0, 13.1}, {1.4, 0, 0, 0}},
    {3, 4, 1, {{1.20, 0, 0, 0}, {2.17, 0, 0, 0}}, {10.0, 13.1}, {1.4, 0, 0, 0}},
    {2, 2, 2, {{0.64, 0.88, 0, 0}, {0.90, 1.64, 0, 0}}, {4.0, 6.0}, {1.10, 1.30, 0, 0}},
    {1, 1, 4, {{0.28, 0.44, 0.62, 0.79}, {0.40, 0.58, 0.85, 1.12}}, {3.5, 4.0}, {0.72, 0.97, 1.2, 1.4}},
};

}  // namespace

// The plan with the least time by the table: full rounds of workgroups over the
// CUs, then the rest.  What decides is how the tiles fill the last round
// (2048 x 6144 x 8192 to fp32: 192 tiles of 256 x 256 take 192 us, 256 of 256 x
// 192 take 155), for few tiles whether splitting a long contraction repays its
// second launch and the partial sums' traffic (128 x 16384 x 8192: 40 us split by 4,
// 56 whole; 1000 x 777 x 1500: 9.3 us whole, 14 us split by 2), and whether the
// product is small enough for the narrow kernels.
MatmulPlan muonh::plan_block_matmul(int c_bf16, const BlockMatmulArgs& a) {
  const int64_t m = a.m, n = a.n, nk = a.kblocks;
  MatmulPlan best{0, 0, 1, a.kblocks, 0};
  // Up to 16 rows (or columns) are narrow: the other operand is read once, at HBM's
  // rate (16 x 12288 x 16384: 42 us, 50 in tiles).  Tiles need panels of 256 rows
  // of values and of scales below 2^31 bytes (buffer offsets).
  const int64_t most = (int64_t)1 << 23;
  if (nk == 0 || m <= 16 || n <= 16 || a.lda >= most || a.ldb >= most || a.ldsa >= most || a.ldsb >= most)
    return best;
  const int arith = c_bf16 ? 0 : 1;
  // Narrow for more rows, in 16 x 16 outputs that each read their 32 rows: measured
  // time of a block per workgroup on each CU (at least the latency of its share).
  // 32 x 2048 x 2048: 3.6 us, 7.1 in tiles; 64 x 512 x 6144: 4.4 and 9.8.  One price
  // of operands beyond L2 per tile shape (`cold`) is too high for some long operands
  // of few tile rows, which go narrow where tiles are quicker: 48 x 12288 x 2048 13.5
  // us (11.0), 32 x 6144 x 16384 34.1 (26.6), 64 x 6144 x 6144 17.2 (15.3).
  const double per_cu = (double)(ceil_div(m, 16) * ceil_div(n, 16)) / kCus;
  double best_us = narrow_direct(a) ? 2.6 + 0.14 * nk * per_cu : 2.5 + nk * std::max(0.045, 0.066 * per_cu);
  for (const TileRate& r : kTileRates) {
    const int64_t mt = ceil_div(m, 64 * r.ma), nt = ceil_div(n, 64 * r.nb), tiles = mt * nt;
    const bool cold = (m + n) * nk * kFp8Block >= kColdBytes && std::min(mt, nt) <= 4;
    auto block_us = [&](int64_t per) { return std::max(r.block[arith][per - 1], cold ? r.cold[per - 1] : 0.0); };
    for (int64_t splits = 1; splits <= 16; splits *= 2) {
      // whole scale words (4 blocks) per workgroup, at least 4 blocks
      const int64_t blocks = splits == 1 ? nk : ceil_div(ceil_div(nk, splits), 4) * 4;
      const int64_t used = ceil_div(nk, blocks), groups = tiles * used;
      if (splits > 1 && (used < 2 || groups > 2 * kCus * r.per_cu)) break;
      const int64_t full = groups / (kCus * r.per_cu), rest = groups - full * kCus * r.per_cu;
      double us = full * (block_us(r.per_cu) * blocks + r.round[arith]);
      if (rest > 0) us += block_us(ceil_div(rest, kCus)) * blocks + r.round[arith];
      // a launch, a workspace, and partials written and read at about 4 TB/s
      if (used > 1) us += 6.0 + (double)((2 * used + 1) * m * n) * 4.0 / 4e6;
      if (us < best_us) {
        best_us = us;
        best = MatmulPlan{r.ma, r.nb, (int32_t)used, (int32_t)blocks,
                          used > 1 ? sizeof(float) * (size_t)(used * m * n) : 0};
      }
    }
  }
  return best;
}

extern "C" {

int muonh_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                         const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt, void* stream) {
  return guarded([&]() -> int {
    int rc;
    if (!q && !qt) return fail(MUONH_EINVAL, "neither form is asked for");
    if ((rc = check_dtype(dtype, "x"))) return rc;
    if ((rc = check_size(rows, 0, "rows")) || (rc = check_size(cols, 0, "cols"))) return rc;
    if ((rc = check_pitch(ldx, rows, cols, "ldx"))) return rc;
    if (q) {
      if ((rc = check_fp8_matrix(*q, "q"))) return rc;
      if (q->rows != rows || q->cols != cols) return fail(MUONH_EINVAL, "q: shape differs from x");
    }
    if (qt) {
      if ((rc = check_fp8_matrix(*qt, "qt"))) return rc;
      if (qt->rows != cols || qt->cols != rows) return fail(MUONH_EINVAL, "qt: shape differs from x transposed");
    }
    if (q && qt && q->block_rows != qt->block_rows) return fail(MUONH_EINVAL, "q and qt: block_rows differ");
    if (rows == 0 || cols == 0) return MUONH_OK;
    const int64_t size = dtype == MUONH_BF16 ? 2 : 4, nx = extent(rows, cols, ldx, size);
    if (!x) return fail(MUONH_EINVAL, "null x");
    if (!aligned(x, (uintptr_t)size)) return fail(MUONH_EINVAL, "misaligned x");
    for (const muonh_fp8_matrix* m : {q, qt})
      if (m && (fp8_overlaps(*m, x, nx) || overlap(m->scale, fp8_scale_bytes(*m), m->data, fp8_data_bytes(*m))))
        return fail(MUONH_EINVAL, "outputs overlap x or each other");
    if (q && qt && (fp8_overlaps(*q, qt->data, fp8_data_bytes(*qt)) || fp8_overlaps(*q, qt->scale, fp8_scale_bytes(*qt))))
      return fail(MUONH_EINVAL, "outputs overlap x or each other");
    if (ceil_div(rows, kFp8Tile) * ceil_div(cols, kFp8Tile) * kQuantizeThreads > kMaxThreads)
      return fail(MUONH_EINVAL, "x is too large for one launch");
    QuantArgs a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    if (q) set_row_form(a, *q);
    if (qt) set_column_form(a, *qt);
    const int32_t block = q ? q->block_rows : qt->block_rows;
    forget_older_errors();
    return launched(launch_block_quantize(dtype == MUONH_BF16, block == 128, a,
                                          reinterpret_cast<hipStream_t>(stream)),
                    "block_quantize");
  });
}

int muonh_block_matmul_workspace(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, int32_t c_dtype,
                                 size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_operands(a, b)) || (rc = check_dtype(c_dtype, "c"))) return rc;
    *bytes = plan_block_matmul(c_dtype == MUONH_BF16, matmul_args(*a, *b)).workspace_bytes;
    return MUONH_OK;
  });
}

int muonh_block_matmul(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, void* c, int32_t c_dtype,
                       int64_t ldc, int32_t accumulate, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return guarded([&]() -> int {
    int rc;
    if ((rc = check_operands(a, b)) || (rc = check_dtype(c_dtype, "c"))) return rc;
    if ((rc = check_pitch(ldc, a->rows, b->rows, "ldc"))) return rc;
    if (accumulate != 0 && accumulate != 1) return fail(MUONH_EINVAL, "accumulate must be 0 or 1");
    if (a->rows == 0 || b->rows == 0) return MUONH_OK;
    const int64_t size = c_dtype == MUONH_BF16 ? 2 : 4, nc = extent(a->rows, b->rows, ldc, size);
    if (!c) return fail(MUONH_EINVAL, "null c");
    if (!aligned(c, (uintptr_t)size)) return fail(MUONH_EINVAL, "misaligned c");
    for (const muonh_fp8_matrix* m : {a, b})
      if (fp8_overlaps(*m, c, nc))
        return fail(MUONH_EINVAL, "c overlaps an operand");
    BlockMatmulArgs p = matmul_args(*a, *b);
    p.c = c;
    p.ldc = ldc;
    p.accumulate = accumulate;
    const MatmulPlan plan = plan_block_matmul(c_dtype == MUONH_BF16, p);
    const int64_t tile_a = plan.ma ? 64 * plan.ma : 16, tile_b = plan.ma ? 64 * plan.nb : 16;
    if (ceil_div(p.m, tile_a) * ceil_div(p.n, tile_b) * plan.splits * 256 > kMaxThreads)
      return fail(MUONH_EINVAL, "c is too large for one launch");
    if (plan.workspace_bytes > 0 && (!workspace || workspace_bytes < plan.workspace_bytes))
      return fail(MUONH_ENOMEM, "workspace too small: need " + std::to_string(plan.workspace_bytes) + " bytes");
    if (!aligned(workspace, kAlign)) return fail(MUONH_EINVAL, "workspace must be 256-byte aligned");
    const int64_t nws = (int64_t)plan.workspace_bytes;
    if (overlap(workspace, nws, c, nc) || fp8_overlaps(*a, workspace, nws) || fp8_overlaps(*b, workspace, nws))
      return fail(MUONH_EINVAL, "workspace overlaps c or an operand");
    forget_older_errors();
    return launched(launch_block_matmul(c_dtype == MUONH_BF16, plan, p, static_cast<float*>(workspace),
                                        reinterpret_cast<hipStream_t>(stream)),
                    "block_matmul");
  });
}

int muonh_norm_forward(const muonh_norm_args* g, void* stream) {
  return guarded([&]() -> int {
    int rc;
    if (!g) return fail(MUONH_EINVAL, "null argument");
    if ((rc = check_dtype(g->dtype, "x"))) return rc;
    if (g->kind != MUONH_NORM_LAYER && g->kind != MUONH_NORM_RMS) return fail(MUONH_EINVAL, "unknown norm kind");
    if (g->reserved != 0) return fail(MUONH_EINVAL, "reserved != 0");
    if (!(g->eps >= 0.0f) || !std::isfinite(g->eps)) return fail(MUONH_EINVAL, "eps must be >= 0 and finite");
    if ((rc = check_norm_size(g->rows, g->cols))) return rc;
    if ((rc = check_pitch(g->ldx, g->rows, g->cols, "ldx")) || (rc = check_pitch(g->ldy, g->rows, g->cols, "ldy"))) return rc;
    const int layer = g->kind == MUONH_NORM_LAYER;
    if (!layer && g->mean) return fail(MUONH_EINVAL, "mean must be NULL for MUONH_NORM_RMS");
    if (g->rows == 0) return MUONH_OK;
    if ((rc = check_vectors(g->x && g->y && g->weight && g->rstd && (!layer || g->mean), "x, y, weight, rstd or mean")))
      return rc;
    const int64_t size = g->dtype == MUONH_BF16 ? 2 : 4;
    if (!aligned(g->x, (uintptr_t)size) || !aligned(g->y, (uintptr_t)size) || !aligned(g->weight, 4) ||
        !aligned(g->bias, 4) || !aligned(g->mean, 4) || !aligned(g->rstd, 4))
      return fail(MUONH_EINVAL, "misaligned pointer");
    if (!may_share(g->y, g->ldy, g->x, g->ldx, g->rows, g->cols, size))
      return fail(MUONH_EINVAL, "y overlaps x");
    const Span x{g->x, extent(g->rows, g->cols, g->ldx, size)}, y{g->y, extent(g->rows, g->cols, g->ldy, size)};
    const Span mean = vec(g->mean, g->rows), rstd = vec(g->rstd, g->rows);
    if (clash({y, mean, rstd}, {vec(g->weight, g->cols), vec(g->bias, g->cols)}) || clash({mean, rstd}, {x}))
      return fail(MUONH_EINVAL, "an output overlaps an input or another output");
    NormArgs a{};
    a.x = g->x;
    a.weight = g->weight;
    a.bias = g->bias;
    a.y = g->y;
    a.mean = g->mean;
    a.rstd = g->rstd;
    a.rows = g->rows;
    a.cols = g->cols;
    a.ldx = g->ldx;
    a.ldy = g->ldy;
    a.eps = g->eps;
    forget_older_errors();
    return launched(launch_norm_forward(g->dtype == MUONH_BF16, layer, a, reinterpret_cast<hipStream_t>(stream)),
                    "norm_forward");
  });
}

int muonh_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_norm_size(rows, cols))) return rc;
    *bytes = (size_t)(2 * norm_partial_rows(rows, cols) * cols) * sizeof(float);
    return MUONH_OK;
  });
}

int muonh_norm_backward(const muonh_norm_grad_args* g, void* stream) {
  return guarded([&]() -> int {
    int rc;
    if (!g) return fail(MUONH_EINVAL, "null argument");
    if ((rc = check_dtype(g->dtype, "x"))) return rc;
    if (g->kind != MUONH_NORM_LAYER && g->kind != MUONH_NORM_RMS) return fail(MUONH_EINVAL, "unknown norm kind");
    if (g->reserved != 0) return fail(MUONH_EINVAL, "reserved != 0");
    if (g->accumulate != 0 && g->accumulate != 1) return fail(MUONH_EINVAL, "accumulate must be 0 or 1");
    if ((rc = check_norm_size(g->rows, g->cols))) return rc;
    if ((rc = check_pitch(g->ld_dy, g->rows, g->cols, "ld_dy")) || (rc = check_pitch(g->ldx, g->rows, g->cols, "ldx")) ||
        (rc = check_pitch(g->ld_dx, g->rows, g->cols, "ld_dx")))
      return rc;
    const int layer = g->kind == MUONH_NORM_LAYER;
    if (!layer && g->mean) return fail(MUONH_EINVAL, "mean must be NULL for MUONH_NORM_RMS");
    if ((rc = check_vectors(g->weight && g->dweight, "weight or dweight"))) return rc;
    const int64_t size = g->dtype == MUONH_BF16 ? 2 : 4;
    if (g->rows > 0) {
      if ((rc = check_vectors(g->dy && g->x && g->dx && g->rstd && (!layer || g->mean), "dy, x, dx, rstd or mean")))
        return rc;
      if (!aligned(g->dy, (uintptr_t)size) || !aligned(g->x, (uintptr_t)size) || !aligned(g->dx, (uintptr_t)size))
        return fail(MUONH_EINVAL, "misaligned pointer");
      if (!may_share(g->dx, g->ld_dx, g->dy, g->ld_dy, g->rows, g->cols, size) ||
          !may_share(g->dx, g->ld_dx, g->x, g->ldx, g->rows, g->cols, size))
        return fail(MUONH_EINVAL, "dx overlaps dy or x");
    }
    if (!aligned(g->weight, 4) || !aligned(g->mean, 4) || !aligned(g->rstd, 4) || !aligned(g->dweight, 4) ||
        !aligned(g->dbias, 4))
      return fail(MUONH_EINVAL, "misaligned pointer");
    size_t need = 0;
    if ((rc = muonh_norm_backward_workspace(g->rows, g->cols, &need))) return rc;
    if (need > 0 && (!g->workspace || g->workspace_bytes < need))
      return fail(MUONH_ENOMEM, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned(g->workspace, kAlign)) return fail(MUONH_EINVAL, "workspace must be 256-byte aligned");
    const Span dy{g->dy, extent(g->rows, g->cols, g->ld_dy, size)}, x{g->x, extent(g->rows, g->cols, g->ldx, size)};
    const Span dx{g->dx, extent(g->rows, g->cols, g->ld_dx, size)}, ws{g->workspace, (int64_t)need};
    const Span dweight = vec(g->dweight, g->cols), dbias = vec(g->dbias, g->cols);
    if (clash({dx, dweight, dbias, ws}, {vec(g->weight, g->cols), vec(g->mean, g->rows), vec(g->rstd, g->rows)}) ||
        clash({dweight, dbias, ws}, {dy, x}))
      return fail(MUONH_EINVAL, "an output or the workspace overlaps an input or another output");
    NormGradArgs a{};
    a.dy = g->dy;
    a.x = g->x;
    a.weight = g->weight;
    a.mean = g->mean;
    a.rstd = g->rstd;
    a.dx = g->dx;
    a.dweight = g->dweight;
    a.dbias = g->dbias;
    a.partials = static_cast<float*>(g->workspace);
    a.rows = g->rows;
    a.cols = g->cols;
    a.lddy = g->ld_dy;
    a.ldx = g->ldx;
    a.lddx = g->ld_dx;
    a.accumulate = g->accumulate;
    forget_older_errors();
    return launched(launch_norm_backward(g->dtype == MUONH_BF16, layer, a, reinterpret_cast<hipStream_t>(stream)),
                    "norm_backward");
  });
}

}  // extern "C"
