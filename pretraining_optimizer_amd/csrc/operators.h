// Launchers of the block-scaled FP8 operators (block_fp8.hip) and of the norms
// (norm.hip), and the checks their C entry points share.  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <exception>
#include <string>

#include "internal.h"

namespace muonh {

constexpr int kFp8Block = 128;   // elements of the contraction that share a scale
constexpr int kFp8Tile = 128;    // the quantiser's tile: 128 x 128 elements per workgroup
constexpr int kQuantizeThreads = 512;

// The quantiser's view of one matrix: x [rows x cols], and the outputs of its
// row form (q, s) and of its column form (qt, st); a null q or qt is not written.
struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t* q;
  uint8_t* s;
  int64_t ldq, lds;
  uint8_t* qt;
  uint8_t* st;
  int64_t ldqt, ldst;
};
// bf16: x's type; square: blocks of 128 x 128 (else 1 x 128).
hipError_t launch_block_quantize(int bf16, int square, const QuantArgs& a, hipStream_t st);

// One workgroup of the step that also quantises: tile (tr, tc) of matrix mat.
struct StepTile {
  int32_t mat;
  uint32_t tr, tc;
};
// The update W <- k1 W - k2 u of every tile, and the forms outs[mat] names (x and
// ldx unused).  bf16: the type of u.
hipError_t launch_update_quantize(int bf16, const StepTile* tiles, int64_t ntiles, const QuantArgs* outs,
                                  const MatGeom* geo, const MatPtrs* ptrs, const MatScalars* scal, hipStream_t st);

constexpr int64_t kCus = 256;   // of an MI355X

// C[m][n] (+)= sum_k A[m][k] B[n][k].
struct BlockMatmulArgs {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* sa;
  const uint8_t* sb;
  int64_t lda, ldb, ldsa, ldsb;   // bytes
  void* c;
  int64_t ldc;                    // elements
  int32_t m, n, kblocks;          // kblocks: blocks of 128 along the contraction
  int32_t a_shift, b_shift;       // scale row = row >> shift (0 or 7)
  int32_t accumulate;
  // Set by the launcher: workgroups along the contraction, blocks of each.
  int32_t splits, split_blocks;
};

// Whether a narrow product's operands go straight into registers, not through
// LDS.  There 16 rows' offsets have to fit 31 bits, and 2^22 workgroups a launch.
// Short contractions are quicker without (1 x 12288 x 1024: 5.0 us, 5.7 through LDS;
// 16 x 6144 x 1024: 4.8 and 4.2; 1 x 6144 x 512: 2.8 and 3.4; 1 x 37984 x 2048: 16.6
// and 17.9, 16 rows of it 25 and 20).
inline bool narrow_direct(const BlockMatmulArgs& a) {
  const int64_t tiles = (((int64_t)a.m + 15) / 16) * (((int64_t)a.n + 15) / 16);
  const int32_t least = a.m < a.n ? a.m : a.n;
  return a.lda >= (1 << 27) || a.ldb >= (1 << 27) || tiles > (1 << 22) || a.kblocks < 8 ||
         (a.kblocks < (least <= 2 ? 32 : 16) && tiles > 2 * kCus);
}

// How a product runs: 64 ma x 64 nb tiles (ma = 0: a narrow kernel), the
// contraction split over `splits` workgroups of split_blocks blocks each, whose
// partial matrices then take workspace_bytes.
struct MatmulPlan {
  int32_t ma, nb, splits, split_blocks;
  size_t workspace_bytes;
};
MatmulPlan plan_block_matmul(int c_bf16, const BlockMatmulArgs& a);
hipError_t launch_block_matmul(int c_bf16, const MatmulPlan& plan, const BlockMatmulArgs& a, float* workspace,
                               hipStream_t st);

struct NormArgs {
  const void* x;
  const float* weight;
  const float* bias;    // nullable
  void* y;
  float* mean;          // layer norm only
  float* rstd;
  int64_t rows, cols, ldx, ldy;
  float eps;
};
hipError_t launch_norm_forward(int bf16, int layer, const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const void* dy;
  const void* x;
  const float* weight;
  const float* mean;    // layer norm only
  const float* rstd;
  void* dx;
  float* dweight;
  float* dbias;         // nullable
  float* partials;      // norm_partial_rows() rows of cols floats (twice that with dbias)
  int64_t rows, cols, lddy, ldx, lddx;
  int32_t accumulate;
  const void* dh;       // launch_add_norm_backward only: added to dx
  int64_t lddh;
};
// Rows of per-workgroup partial sums of dweight that a backward pass writes.
int64_t norm_partial_rows(int64_t rows, int64_t cols);
hipError_t launch_norm_backward(int bf16, int layer, const NormGradArgs& a, hipStream_t st);

// The residual's addition, the RMS norm of the sum and its FP8 forms: first h, rstd
// and, of rows that registers hold (add_norm_rows_quantize), the row form, then the
// other forms of h rstd weight, tile by tile.
struct AddNormArgs {
  const void* x;
  const void* residual;   // nullable: h is x, and not written
  const float* weight;
  void* h;
  float* rstd;
  int64_t rows, cols, ldx, ldr, ldh;
  float eps;
  uint8_t* q;             // nullable: the row form is not written here
  uint8_t* s;
  int64_t ldq, lds;
};
bool add_norm_rows_quantize(int64_t cols);
hipError_t launch_add_norm_rows(int bf16, const AddNormArgs& a, hipStream_t st);
// out.x, out.ldx: h.
hipError_t launch_norm_quantize(int bf16, const QuantArgs& out, const float* weight, const float* rstd, hipStream_t st);
// norm_backward of an RMS norm without bias, whose dx also takes dh.
hipError_t launch_add_norm_backward(int bf16, const NormGradArgs& a, hipStream_t st);

// Checks one FP8 operand; `whose` names it in the error text.
int check_fp8_matrix(const muonh_fp8_matrix& m, const char* whose);
// Its forms' addresses in QuantArgs.
void set_row_form(QuantArgs& a, const muonh_fp8_matrix& m);
void set_column_form(QuantArgs& a, const muonh_fp8_matrix& m);
// Bytes of a row's values and scales with their padding, and from the first to
// behind the last of all rows.
int64_t fp8_data_width(const muonh_fp8_matrix& m);
int64_t fp8_scale_width(const muonh_fp8_matrix& m);
int64_t fp8_data_bytes(const muonh_fp8_matrix& m);
int64_t fp8_scale_bytes(const muonh_fp8_matrix& m);
// Whether an operand's values or scales share memory with [p, p + bytes).
bool fp8_overlaps(const muonh_fp8_matrix& m, const void* p, int64_t bytes);

// HIP keeps a failed call's error until it is read, and a launch's own is read the
// same way: one that the thread left behind earlier (an allocation that it gave up
// on) would be taken for the launch's.
inline void forget_older_errors() { (void)hipGetLastError(); }

// Runs the body of a C entry point; nothing is thrown across the ABI.
template <typename F>
int guarded(F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      return set_last_error(MUONH_ENOMEM, e.what());
    } catch (...) {
      return MUONH_ENOMEM;
    }
  }
}

}  // namespace muonh
