// Layer norm and RMS norm over the last axis, and their gradients (gfx950).
//
//   layer: mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), h = (x - mu) r
//   rms:   r = 1 / sqrt(mean(x^2) + eps),                      h = x r
//   y = h w (+ b)
//   g = dy w;  dx = r (g - [mean(g)] - h mean(g h))            ([]: layer only)
//   dw = sum over rows of dy h;  db = sum over rows of dy
//
// Both passes are bound by HBM: forward reads x and writes y, backward reads
// x and dy and writes dx.  A row is held in registers between its reduction
// and its output, so each of these streams passes once; the variance is taken
// about the mean of the values in hand, not from a difference of moments.
// Statistics, sums and the weight gradient are fp32; each output element is
// rounded once.  8192 x 2048 bf16, calls in a row: forward 12.8 us (5.2 TB/s, part of
// it from the 256 MB cache), backward with the partial rows' sum 21.8 us (4.6 TB/s).
// Loads and stores are ordinary ones: the input was just written by another
// operator and the output is read by the next (8192 x 2048 fp32 forward: 27.4 us,
// 32.3 with non-temporal accesses).

#include <algorithm>

#include "fp8_convert.h"
#include "operators.h"
#include "row_vectors.h"

namespace muonh {
namespace {

constexpr int kNormThreads = 256;
// Workgroups of a backward pass, one per CU: each adds its rows' dy h in
// registers and leaves one row of partial sums, which a second launch adds in
// order.
constexpr int kNormGroups = 256;
constexpr int kBackThreads = 512;

// A weight or bias vector: read by every row, so through the caches.
__device__ __forceinline__ void loadw(const float* w, int c, int n, float (&v)[8]) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  if (c + 8 <= n) {
    const vec lo = ld_global<vec>(w + c), hi = ld_global<vec>(w + c + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = lo[k];
      v[4 + k] = hi[k];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < n ? ld_global<float>(w + c + j) : 0.0f;
  }
}

// v rounded to T, as fp32.
template <typename T>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(f32_to_bf16(v));
  else return v;
}

// Sums of NS values over the G threads of a row, the same in each of them: a
// shuffle tree inside a wavefront, and the wavefronts' sums in order through
// LDS for longer groups (every thread of the workgroup then takes part).
template <int G, int NS>
__device__ __forceinline__ void group_sum(float (&s)[NS], float (*red)[16]) {
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int off = (G < 64 ? G : 64) / 2; off > 0; off >>= 1) s[k] += __shfl_xor(s[k], off, 64);
  if constexpr (G > 64) {
    __syncthreads();   // the previous reduction's sums have been read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < NS; ++k) red[k][threadIdx.x >> 6] = s[k];
    }
    __syncthreads();
    const int w0 = (threadIdx.x / G) * (G / 64);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      s[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) s[k] += red[k][w0 + w];
    }
  }
}

// A group of G threads per row, NV vectors of 8 elements per thread: thread t
// of a group holds elements 8 (t + G k) .. + 7.  8 G NV >= cols.
template <typename T, bool LAYER, int G, int NV>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void norm_forward_kernel(NormArgs p) {
  constexpr int kThreads = G > kNormThreads ? G : kNormThreads;
  constexpr int kRows = kThreads / G;
  __shared__ float red[1][16];
  const int t = threadIdx.x % G, cols = (int)p.cols;
  const float rn = 1.0f / (float)cols;
  // Every thread of the workgroup takes each trip, so the barriers inside
  // group_sum are met by all of them.
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + threadIdx.x / G;
    const bool live = row < p.rows;
    const T* x = reinterpret_cast<const T*>(p.x) + (live ? row : p.rows - 1) * p.ldx;
    float v[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) load8<T>(x, 8 * (t + G * k), cols).widen(v[k]);
    float mu = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += v[k][j];
      group_sum<G, 1>(s, red);
      mu = s[0] * rn;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 8 * (t + G * k) + j < cols ? v[k][j] - mu : 0.0f;
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += v[k][j] * v[k][j];
    group_sum<G, 1>(ss, red);
    const float r = 1.0f / sqrtf(ss[0] * rn + p.eps);
    if (!live) continue;
    if (t == 0) {
      if constexpr (LAYER) p.mean[row] = mu;
      p.rstd[row] = r;
    }
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (t + G * k);
      if (c >= cols) continue;
      float w[8], b[8];
      loadw(p.weight, c, cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = v[k][j] * r * w[j];
      if (p.bias) {
        loadw(p.bias, c, cols, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += b[j];
      }
      store8<T>(y, c, cols, w);
    }
  }
}

// h = x + residual, kept in x's type, 1 / sqrt(mean(h^2) + eps) of the kept values, and
// the row form of y = (h r) w in block-scaled FP8, all from the registers that hold the
// row: 16 threads have a group of 128 columns.  y is rounded once, to E4M3.  Without a
// residual h is x, which is only read.  Bound by HBM: 8192 x 2048 bf16 with a residual
// 23 us, 5.1 TB/s, as a copy.
template <typename T, int G, int NV>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void add_norm_rows_kernel(AddNormArgs p) {
  static_assert(G >= 16, "16 threads share a scale");
  constexpr int kThreads = G > kNormThreads ? G : kNormThreads;
  constexpr int kRows = kThreads / G;
  __shared__ float red[1][16];
  const int t = threadIdx.x % G, cols = (int)p.cols;
  const int groups = (cols + kFp8Block - 1) / kFp8Block;
  const float rn = 1.0f / (float)cols;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + threadIdx.x / G, at = min(row, p.rows - 1);
    const bool live = row < p.rows;
    const T* x = reinterpret_cast<const T*>(p.x) + at * p.ldx;
    const T* r = reinterpret_cast<const T*>(p.residual) + at * p.ldr;
    float v[NV][8];
    {
      Raw8<T> a[NV], b[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        a[k] = load8<T>(x, 8 * (t + G * k), cols);
        if (p.residual) b[k] = load8<T>(r, 8 * (t + G * k), cols);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        a[k].widen(v[k]);
        if (p.residual) {
          float w[8];
          b[k].widen(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] = round_to<T>(v[k][j] + w[j]);
          const int c = 8 * (t + G * k);
          if (live && c < cols) store8<T>(reinterpret_cast<T*>(p.h) + row * p.ldh, c, cols, v[k]);
        }
      }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += v[k][j] * v[k][j];
    group_sum<G, 1>(ss, red);
    const float rstd = 1.0f / sqrtf(ss[0] * rn + p.eps);
    if (live && t == 0) p.rstd[row] = rstd;
    if (!p.q) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (t + G * k), group = c / kFp8Block;
      float w[8];
      loadw(p.weight, c, cols, w);
      // behind the end 0 r w is no zero where r or w is infinite
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = c + j < cols ? v[k][j] * rstd * w[j] : 0.0f;
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(v[k][j]) & 0x7fffffffu);
      const bool special = most >= 0x7f800000u;
      if (special) {
        most = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t m = __float_as_uint(v[k][j]) & 0x7fffffffu;
          most = max(most, m < 0x7f800000u ? m : 0u);
        }
      }
      const uint32_t byte = scale_byte(max16(most));
      u32x2_t q;
      if (special) {
        q[0] = pack_fp8(scaled(v[k][0], byte), scaled(v[k][1], byte), scaled(v[k][2], byte), scaled(v[k][3], byte));
        q[1] = pack_fp8(scaled(v[k][4], byte), scaled(v[k][5], byte), scaled(v[k][6], byte), scaled(v[k][7], byte));
      } else {
        const float scale = __uint_as_float(byte << 23);
        q[0] = quantize4(v[k][0], v[k][1], v[k][2], v[k][3], scale);
        q[1] = quantize4(v[k][4], v[k][5], v[k][6], v[k][7], scale);
      }
      if (!live || group >= groups) continue;
      st_global<u32x2_t>(p.q + row * p.ldq + c, q);   // zeros up to the group's end
      if ((t & 15) == 0) {
        uint8_t* s = p.s + row * p.lds + group;
        *s = (uint8_t)byte;
        if (group == groups - 1)   // zero bytes up to a multiple of 4
          for (int z = groups; z & 3; ++z) p.s[row * p.lds + z] = 0;
      }
    }
  }
}

// Rows too long for registers: one workgroup per row reads it once per
// reduction and once for the output, from the caches after the first.
//
// A thread adds kLongRun terms in fp32 and those sums in fp64, so a row of any
// length is summed as exactly as one that fits registers (one fp32 chain over the
// 4096 terms of 2^22 columns is off by 4e-5).  Bound by the latency of accesses of
// one element each: 512 x 20000 bf16 takes 17.8 us forward and 48.9 backward (2.3
// and 1.3 TB/s), 8 x 65536 35 and 48 us.
constexpr int kLongThreads = 1024;
constexpr int kLongRun = 32;
template <typename F>
__device__ __forceinline__ float long_sum(int64_t cols, F term) {
  double total = 0.0;
  for (int64_t c0 = threadIdx.x; c0 < cols; c0 += kLongThreads * kLongRun) {
    const int64_t end = min(cols, c0 + kLongThreads * kLongRun);
    float s = 0.0f;
    for (int64_t c = c0; c < end; c += kLongThreads) s += term(c);
    total += (double)s;
  }
  return (float)total;
}

template <typename T, bool LAYER>
__global__ __launch_bounds__(kLongThreads) void norm_forward_long_kernel(NormArgs p) {
  __shared__ float red[1][16];
  const double rn = 1.0 / (double)p.cols;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
    float mu = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {long_sum(p.cols, [&](int64_t c) { return Raw8<T>::load1(x + c); })};
      group_sum<kLongThreads, 1>(s, red);
      mu = (float)((double)s[0] * rn);
    }
    float ss[1] = {long_sum(p.cols, [&](int64_t c) {
      const float d = Raw8<T>::load1(x + c) - mu;
      return d * d;
    })};
    group_sum<kLongThreads, 1>(ss, red);
    const float r = 1.0f / sqrtf((float)((double)ss[0] * rn) + p.eps);
    if (threadIdx.x == 0) {
      if constexpr (LAYER) p.mean[row] = mu;
      p.rstd[row] = r;
    }
    for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
      float v = (Raw8<T>::load1(x + c) - mu) * r * p.weight[c];
      if (p.bias) v += p.bias[c];
      Raw8<T>::store1(y + c, v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kLongThreads) void add_norm_rows_long_kernel(AddNormArgs p) {
  __shared__ float red[1][16];
  const double rn = 1.0 / (double)p.cols;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    const T* r = reinterpret_cast<const T*>(p.residual) + row * p.ldr;
    T* h = reinterpret_cast<T*>(p.h) + row * p.ldh;
    float ss[1] = {long_sum(p.cols, [&](int64_t c) {
      float v = Raw8<T>::load1(x + c);
      if (p.residual) {
        v = round_to<T>(v + Raw8<T>::load1(r + c));
        Raw8<T>::store1(h + c, v);
      }
      return v * v;
    })};
    group_sum<kLongThreads, 1>(ss, red);
    if (threadIdx.x == 0) p.rstd[row] = 1.0f / sqrtf((float)((double)ss[0] * rn) + p.eps);
  }
}

// Backward.  Workgroup b takes rows kRows b .. , kRows (b + gridDim.x) .. and
// so on; a thread keeps the same columns for all of its rows and adds dy h
// (and dy) for them in registers.  At the end the groups of one workgroup are
// added in order through LDS, and the workgroup writes one row of partials.
// RES: dx also takes the residual stream's gradient dh, rounded once.
template <typename T, bool LAYER, bool BIAS, bool RES, int G, int NV>
__global__ __launch_bounds__(G > kBackThreads ? G : kBackThreads) void norm_backward_kernel(NormGradArgs p) {
  constexpr int kThreads = G > kBackThreads ? G : kBackThreads;
  constexpr int kRows = kThreads / G;
  constexpr int kAcc = BIAS ? 2 : 1;
  __shared__ float red[2][16];
  __shared__ __attribute__((aligned(16))) float fold[kRows > 1 ? kThreads * 8 : 1];
  const int t = threadIdx.x % G, grp = threadIdx.x / G, cols = (int)p.cols;
  const float rn = 1.0f / (float)cols;
  const int64_t step = (int64_t)gridDim.x * kRows;
  // The next trip's rows are on their way while this one's are used, and the
  // weight stays in registers; 1024 threads have no room for either.
  constexpr bool kAhead = kThreads < 1024;
  Raw8<T> nx[NV], nd[NV], nh[RES ? NV : 1];
  float nr = 0.0f, nmu = 0.0f;
  auto fetch = [&](int64_t r0) {
    const int64_t at = min(r0 + grp, p.rows - 1);
    const T* x = reinterpret_cast<const T*>(p.x) + at * p.ldx;
    const T* dy = reinterpret_cast<const T*>(p.dy) + at * p.lddy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      nx[k] = load8<T>(x, 8 * (t + G * k), cols);
      nd[k] = load8<T>(dy, 8 * (t + G * k), cols);
      if constexpr (RES)
        nh[k] = load8<T>(reinterpret_cast<const T*>(p.dh) + at * p.lddh, 8 * (t + G * k), cols);
    }
    nr = p.rstd[at];
    if constexpr (LAYER) nmu = p.mean[at];
  };
  int64_t r0 = (int64_t)blockIdx.x * kRows;
  if constexpr (kAhead) fetch(r0);
  float w[NV][8], acc[kAcc][NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (kAhead) loadw(p.weight, 8 * (t + G * k), cols, w[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[0][k][j] = 0.0f;
      if constexpr (BIAS) acc[1][k][j] = 0.0f;
    }
  }
  for (; r0 < p.rows; r0 += step) {
    if constexpr (!kAhead) {
      fetch(r0);
#pragma unroll
      for (int k = 0; k < NV; ++k) loadw(p.weight, 8 * (t + G * k), cols, w[k]);
    }
    const int64_t row = r0 + grp;
    const bool live = row < p.rows;
    const float r = nr, mu = nmu;
    float h[NV][8], g[NV][8];
    Raw8<T> dh[RES ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      nx[k].widen(h[k]);
      nd[k].widen(g[k]);
      if constexpr (RES) dh[k] = nh[k];
    }
    if constexpr (kAhead) {
      if (r0 + step < p.rows) fetch(r0 + step);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[k][j] = (h[k][j] - mu) * r;
        // Columns behind the end have no weight gradient to write, and dy = w = 0;
        // h is 0 there too, as (0 - mu) r may be infinite (rms: x = mu = 0).
        if (LAYER && 8 * (t + G * k) + j >= cols) h[k][j] = 0.0f;
        // a group behind the last row adds nothing
        if (live) {
          acc[0][k][j] += g[k][j] * h[k][j];
          if constexpr (BIAS) acc[1][k][j] += g[k][j];
        }
        g[k][j] *= w[k][j];
        s[0] += g[k][j] * h[k][j];
        s[1] += g[k][j];
      }
    group_sum<G, 2>(s, red);
    if (!live) continue;
    const float c1 = s[0] * rn, c0 = LAYER ? s[1] * rn : 0.0f;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (t + G * k);
      if (c >= cols) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r * (g[k][j] - c0 - h[k][j] * c1);
      if constexpr (RES) {
        float a[8];
        dh[k].widen(a);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += a[j];
      }
      store8<T>(dx, c, cols, o);
    }
  }
  // Vector k of the groups covers columns 8 G k .. 8 G (k + 1) - 1.
  float* out = p.partials + (int64_t)blockIdx.x * cols;
#pragma unroll
  for (int a = 0; a < kAcc; ++a) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (kRows > 1) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<f32x4_t*>(&fold[(grp * G + t) * 8 + 4 * h]) =
              f32x4_t{acc[a][k][4 * h], acc[a][k][4 * h + 1], acc[a][k][4 * h + 2], acc[a][k][4 * h + 3]};
        __syncthreads();
        for (int c = threadIdx.x; c < 8 * G; c += kThreads) {
          float v = 0.0f;
#pragma unroll
          for (int q = 0; q < kRows; ++q) v += fold[q * 8 * G + c];
          if (8 * G * k + c < cols) out[8 * G * k + c] = v;
        }
      } else {
        const int c = 8 * (t + G * k);
        typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
        if (c + 8 <= cols) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            st_global<vec>(out + c + 4 * h, vec{acc[a][k][4 * h], acc[a][k][4 * h + 1], acc[a][k][4 * h + 2], acc[a][k][4 * h + 3]});
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < cols) out[c + j] = acc[a][k][j];
        }
      }
    }
    out += (int64_t)gridDim.x * cols;
  }
}

// Rows too long for registers: a workgroup adds each of its rows to its own
// row of partials in memory (each column always by the same thread).
template <typename T, bool LAYER, bool BIAS, bool RES>
__global__ __launch_bounds__(kLongThreads) void norm_backward_long_kernel(NormGradArgs p) {
  __shared__ float red[2][16];
  const double rn = 1.0 / (double)p.cols;
  float* pw = p.partials + (int64_t)blockIdx.x * p.cols;
  float* pb = pw + (int64_t)gridDim.x * p.cols;
  bool first = true;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = reinterpret_cast<const T*>(p.dy) + row * p.lddy;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
    const float r = p.rstd[row], mu = LAYER ? p.mean[row] : 0.0f;
    double total[2] = {0.0, 0.0};
    for (int64_t c0 = threadIdx.x; c0 < p.cols; c0 += kLongThreads * kLongRun) {
      const int64_t end = min(p.cols, c0 + kLongThreads * kLongRun);
      float run[2] = {0.0f, 0.0f};
      for (int64_t c = c0; c < end; c += kLongThreads) {
        const float h = (Raw8<T>::load1(x + c) - mu) * r, d = Raw8<T>::load1(dy + c);
        pw[c] = (first ? 0.0f : pw[c]) + d * h;
        if constexpr (BIAS) pb[c] = (first ? 0.0f : pb[c]) + d;
        const float g = d * p.weight[c];
        run[0] += g * h;
        run[1] += g;
      }
      total[0] += (double)run[0];
      total[1] += (double)run[1];
    }
    float s[2] = {(float)total[0], (float)total[1]};
    first = false;
    group_sum<kLongThreads, 2>(s, red);
    const float c1 = (float)((double)s[0] * rn), c0 = LAYER ? (float)((double)s[1] * rn) : 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
      const float h = (Raw8<T>::load1(x + c) - mu) * r;
      const float g = Raw8<T>::load1(dy + c) * p.weight[c];
      float o = r * (g - c0 - h * c1);
      if constexpr (RES) o += Raw8<T>::load1(reinterpret_cast<const T*>(p.dh) + row * p.lddh + c);
      Raw8<T>::store1(dx + c, o);
    }
  }
}

// dw (and db, blockIdx.y = 1) from the partial rows: 16 columns per workgroup
// and 32 threads per column, each adding every 32nd row, then in order in LDS.
constexpr int kFoldThreads = 512;
__global__ __launch_bounds__(kFoldThreads) void norm_fold_kernel(const float* __restrict__ partials, int64_t nrows,
                                                                 int64_t cols, float* dweight, float* dbias,
                                                                 int accumulate) {
  __shared__ float red[32][17];
  const int lc = threadIdx.x & 15, lr = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + lc;
  const float* p = partials + (blockIdx.y ? nrows * cols : 0);
  float s = 0.0f;
  if (c < cols) {
    float v[kNormGroups / 32];
#pragma unroll
    for (int k = 0; k < kNormGroups / 32; ++k) v[k] = lr + 32 * k < nrows ? p[(lr + 32 * k) * cols + c] : 0.0f;
#pragma unroll
    for (int k = 0; k < kNormGroups / 32; ++k) s += v[k];
  }
  red[lr][lc] = s;
  __syncthreads();
  if (threadIdx.x >= 16 || c >= cols) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) s += red[k][lc];
  float* out = blockIdx.y ? dbias : dweight;
  out[c] = accumulate ? out[c] + s : s;
}

constexpr int64_t kRegisterCols = 16384;   // 1024 threads of 16 elements

// Rows that a workgroup of `threads` takes at a time (the kernels' kRows).
int64_t rows_at_once(int64_t cols, int64_t threads) {
  const int64_t group = cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 1024 ? 64 : cols <= 2048 ? 128
                        : cols <= 4096 ? 256 : cols <= 8192 ? 512 : 1024;
  return std::max<int64_t>(threads / group, 1);
}

template <typename T, bool LAYER>
hipError_t forward_for(const NormArgs& a, hipStream_t st) {
  const int64_t cols = a.cols;
  if (cols > kRegisterCols) {
    hipLaunchKernelGGL((norm_forward_long_kernel<T, LAYER>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)),
                       dim3(kLongThreads), 0, st, a);
    return hipGetLastError();
  }
  const int64_t per = rows_at_once(cols, kNormThreads);
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + per - 1) / per, 1 << 20));
#define MUONH_NORM_FWD(G, NV)                                                                  \
  hipLaunchKernelGGL((norm_forward_kernel<T, LAYER, G, NV>), grid,                             \
                     dim3(G > kNormThreads ? G : kNormThreads), 0, st, a)
  if (cols <= 64) MUONH_NORM_FWD(8, 1);
  else if (cols <= 128) MUONH_NORM_FWD(16, 1);
  else if (cols <= 256) MUONH_NORM_FWD(32, 1);
  else if (cols <= 512) MUONH_NORM_FWD(64, 1);
  else if (cols <= 1024) MUONH_NORM_FWD(64, 2);
  else if (cols <= 2048) MUONH_NORM_FWD(128, 2);
  else if (cols <= 4096) MUONH_NORM_FWD(256, 2);
  else if (cols <= 8192) MUONH_NORM_FWD(512, 2);
  else MUONH_NORM_FWD(1024, 2);
#undef MUONH_NORM_FWD
  return hipGetLastError();
}

template <typename T, bool LAYER, bool BIAS, bool RES = false>
hipError_t backward_for(const NormGradArgs& a, hipStream_t st) {
  const int64_t cols = a.cols, groups = norm_partial_rows(a.rows, cols);
  if (groups > 0) {
    const dim3 grid((unsigned)groups);
#define MUONH_NORM_BWD(G, NV)                                                                  \
  hipLaunchKernelGGL((norm_backward_kernel<T, LAYER, BIAS, RES, G, NV>), grid,                      \
                     dim3(G > kBackThreads ? G : kBackThreads), 0, st, a)
    if (cols > kRegisterCols)
      hipLaunchKernelGGL((norm_backward_long_kernel<T, LAYER, BIAS, RES>), grid, dim3(kLongThreads), 0, st, a);
    else if (cols <= 64) MUONH_NORM_BWD(8, 1);
    else if (cols <= 128) MUONH_NORM_BWD(16, 1);
    else if (cols <= 256) MUONH_NORM_BWD(32, 1);
    else if (cols <= 512) MUONH_NORM_BWD(64, 1);
    else if (cols <= 1024) MUONH_NORM_BWD(64, 2);
    else if (cols <= 2048) MUONH_NORM_BWD(128, 2);
    else if (cols <= 4096) MUONH_NORM_BWD(256, 2);
    else if (cols <= 8192) MUONH_NORM_BWD(512, 2);
    else MUONH_NORM_BWD(1024, 2);
#undef MUONH_NORM_BWD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)((cols + 15) / 16), BIAS ? 2 : 1), dim3(kFoldThreads), 0,
                     st,
                     a.partials, groups, cols, a.dweight, a.dbias, a.accumulate);
  return hipGetLastError();
}

template <typename T>
hipError_t add_norm_rows_for(const AddNormArgs& a, hipStream_t st) {
  const int64_t cols = a.cols;
  if (cols > kRegisterCols) {
    hipLaunchKernelGGL(add_norm_rows_long_kernel<T>, dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)),
                       dim3(kLongThreads), 0, st, a);
    return hipGetLastError();
  }
  const int64_t per = rows_at_once(std::max<int64_t>(cols, 65), kNormThreads);   // groups of 16 threads at least
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + per - 1) / per, 1 << 20));
#define MUONH_ADD_NORM(G, NV)                                                                  \
  hipLaunchKernelGGL((add_norm_rows_kernel<T, G, NV>), grid, dim3(G > kNormThreads ? G : kNormThreads), 0, st, a)
  if (cols <= 128) MUONH_ADD_NORM(16, 1);
  else if (cols <= 256) MUONH_ADD_NORM(32, 1);
  else if (cols <= 512) MUONH_ADD_NORM(64, 1);
  else if (cols <= 1024) MUONH_ADD_NORM(64, 2);
  else if (cols <= 2048) MUONH_ADD_NORM(128, 2);
  else if (cols <= 4096) MUONH_ADD_NORM(256, 2);
  else if (cols <= 8192) MUONH_ADD_NORM(512, 2);
  else MUONH_ADD_NORM(1024, 2);
#undef MUONH_ADD_NORM
  return hipGetLastError();
}

}  // namespace

bool add_norm_rows_quantize(int64_t cols) { return cols <= kRegisterCols; }

hipError_t launch_add_norm_rows(int bf16, const AddNormArgs& a, hipStream_t st) {
  return bf16 ? add_norm_rows_for<uint16_t>(a, st) : add_norm_rows_for<float>(a, st);
}

hipError_t launch_add_norm_backward(int bf16, const NormGradArgs& a, hipStream_t st) {
  return bf16 ? backward_for<uint16_t, false, false, true>(a, st) : backward_for<float, false, false, true>(a, st);
}

int64_t norm_partial_rows(int64_t rows, int64_t cols) {
  const int64_t per = cols > kRegisterCols ? 1 : rows_at_once(cols, kBackThreads);
  const int64_t trips = (rows + per - 1) / per;
  // every workgroup's row of partials is written and read again: at least 2
  // trips each, unless that leaves fewer than 64 workgroups
  return std::min<int64_t>(std::min<int64_t>(trips, std::max<int64_t>(64, (trips + 1) / 2)), kNormGroups);
}

hipError_t launch_norm_forward(int bf16, int layer, const NormArgs& a, hipStream_t st) {
  if (bf16) return layer ? forward_for<uint16_t, true>(a, st) : forward_for<uint16_t, false>(a, st);
  return layer ? forward_for<float, true>(a, st) : forward_for<float, false>(a, st);
}

hipError_t launch_norm_backward(int bf16, int layer, const NormGradArgs& a, hipStream_t st) {
  if (bf16) {
    if (a.dbias) return layer ? backward_for<uint16_t, true, true>(a, st) : backward_for<uint16_t, false, true>(a, st);
    return layer ? backward_for<uint16_t, true, false>(a, st) : backward_for<uint16_t, false, false>(a, st);
  }
  if (a.dbias) return layer ? backward_for<float, true, true>(a, st) : backward_for<float, false, true>(a, st);
  return layer ? backward_for<float, true, false>(a, st) : backward_for<float, false, false>(a, st);
}

}  // namespace muonh
