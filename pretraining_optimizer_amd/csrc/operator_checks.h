// Argument checks that the operators' C entry points share.  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <string>

#include "internal.h"

namespace muonh {

inline int fail(int code, const std::string& msg) { return set_last_error(code, msg.c_str()); }

inline int launched(hipError_t e, const char* what) {
  return e == hipSuccess ? MUONH_OK : fail(MUONH_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;    // row and column counts: tile arithmetic is 32 bits
constexpr int64_t kMaxNormCols = (int64_t)1 << 26;
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;   // of one launch
constexpr size_t kAlign = 256;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int64_t ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Bytes from the first element to behind the last of `rows` rows.
inline int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return rows < 1 || cols < 1 ? 0 : ((rows - 1) * ld + cols) * size;
}

inline bool overlap(const void* p, int64_t pn, const void* q, int64_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return pn > 0 && qn > 0 && a < b + (uintptr_t)qn && b < a + (uintptr_t)pn;
}

struct Span {
  const void* p;
  int64_t bytes;
};
// Whether an output shares memory with another or with an input.
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(o->p, o->bytes, q->p, q->bytes)) return true;
  }
  return false;
}
inline Span vec(const float* p, int64_t n) { return Span{p, p ? n * 4 : 0}; }

// Whether an output may share memory with an input of the same size: in place,
// apart, or in other columns of the same rows.
inline bool may_share(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows, int64_t cols,
               int64_t size) {
  if (!overlap(out, extent(rows, cols, ldo, size), in, extent(rows, cols, ldi, size))) return true;
  if (ldo != ldi && rows > 1) return false;
  if (out == in) return true;
  if (rows == 1) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
  const int64_t d = (int64_t)(a > b ? a - b : b - a) % (ldo * size);
  return d >= cols * size && ldo * size - d >= cols * size;
}

inline int check_dtype(int32_t t, const char* what) {
  if (t != MUONH_F32 && t != MUONH_BF16) return fail(MUONH_EINVAL, std::string(what) + ": dtype must be F32 or BF16");
  return MUONH_OK;
}

inline int check_size(int64_t v, int64_t least, const char* what) {
  if (v < least || v > kMaxRows)
    return fail(MUONH_EINVAL, std::string(what) + " must be in [" + std::to_string(least) + ", 2^30]");
  return MUONH_OK;
}

inline int check_norm_size(int64_t rows, int64_t cols) {
  if (cols < 1 || cols > kMaxNormCols) return fail(MUONH_EINVAL, "cols must be in [1, 2^26]");
  return check_size(rows, 0, "rows");
}

// rows * ld stays at or below 2^60, so a matrix's bytes fit 64 bits.
inline int check_pitch(int64_t ld, int64_t rows, int64_t cols, const char* what) {
  if (ld < cols || ld > ((int64_t)1 << 40) || (rows > 0 && ld > ((int64_t)1 << 60) / rows))
    return fail(MUONH_EINVAL, std::string(what) + ": the pitch is less than a row, or too large");
  return MUONH_OK;
}

}  // namespace muonh
