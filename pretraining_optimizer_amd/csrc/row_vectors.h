// Eight consecutive elements of a matrix row of any alignment and length, for
// the kernels whose threads hold a row between them.
#pragma once

#include "device_util.h"

namespace muonh {

// Eight consecutive elements of a row as stored, from any element alignment
// (global accesses of any width need no more on gfx950), and as fp32.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  vec w;
  __device__ __forceinline__ void load(const uint16_t* p) {
    w = ld_global<vec>(p);
  }
  __device__ __forceinline__ void zero() { w = vec{0, 0, 0, 0}; }
  __device__ __forceinline__ void set(int j, const uint16_t* p) {
    w[j >> 1] |= (uint32_t)ld_global<uint16_t>(p) << (16 * (j & 1));
  }
  // Elements n .. 7 to the front, zeros behind them; 0 < n < 8.
  __device__ __forceinline__ void drop(int n) {
    if (n & 4) w = vec{w[2], w[3], 0, 0};
    if (n & 2) w = vec{w[1], w[2], w[3], 0};
    if (n & 1) w = vec{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(ld_global<uint16_t>(p)); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[8]) {
    vec r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    st_global<vec>(p, r);
  }
  static __device__ __forceinline__ void store1(uint16_t* p, float v) { st_global<uint16_t>(p, f32_to_bf16(v)); }
};
template <> struct Raw8<float> {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  vec lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = ld_global<vec>(p);
    hi = ld_global<vec>(p + 4);
  }
  __device__ __forceinline__ void zero() { lo = hi = vec{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void set(int j, const float* p) {
    const float v = ld_global<float>(p);
    if (j < 4) lo[j] = v;
    else hi[j - 4] = v;
  }
  __device__ __forceinline__ void drop(int n) {
    if (n & 4) {
      lo = hi;
      hi = vec{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (n & 2) {
      lo = vec{lo[2], lo[3], hi[0], hi[1]};
      hi = vec{hi[2], hi[3], 0.0f, 0.0f};
    }
    if (n & 1) {
      lo = vec{lo[1], lo[2], lo[3], hi[0]};
      hi = vec{hi[1], hi[2], hi[3], 0.0f};
    }
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = lo[k];
      v[4 + k] = hi[k];
    }
  }
  static __device__ __forceinline__ float load1(const float* p) { return ld_global<float>(p); }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    st_global<vec>(p, vec{v[0], v[1], v[2], v[3]});
    st_global<vec>(p + 4, vec{v[4], v[5], v[6], v[7]});
  }
  static __device__ __forceinline__ void store1(float* p, float v) { st_global<float>(p, v); }
};

// Elements [c, c + 8) of a row of n, zeros behind its end.  At the end the row's last
// eight are loaded: one by one each load would wait for the one before.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* row, int c, int n) {
  Raw8<T> r;
  if (c + 8 <= n) {
    r.load(row + c);
  } else if (c < n && n >= 8) {
    r.load(row + n - 8);
    r.drop(c + 8 - n);
  } else {
    r.zero();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) r.set(j, row + c + j);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    Raw8<T>::store(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) Raw8<T>::store1(row + c + j, v[j]);
  }
}

}  // namespace muonh
