// Block-scaled FP8 (OCP E4M3 values, power-of-two scales) for gfx950: the
// quantiser of activations, gradients and weights, and the product of two
// quantised operands.
//
// The recipe is the one the pages train the MuonH matrices with ("Puro-2B:
// Poor Lab's Qwen2-1.5B Trained on RTX 5090 within $5090", arXiv HTML §3.2
// and App. C): groups of 1 x 128 along the contraction for activations and
// gradients, blocks of 128 x 128 for weights, power-of-two scales.
//
//   amax = max |x| over the finite elements of a block
//   e    = the least integer with amax <= 448 * 2^e, at least -127 (0 if amax = 0)
//   q    = rne_e4m3(x * 2^-e);   stored scale byte: e + 127 (E8M0)
//
// |x * 2^-e| <= 448, the largest E4M3 value, so a finite element never
// saturates; scaling by a power of two is exact above the subnormals, so the
// only rounding is the one to E4M3.  NaN and Inf become the E4M3 NaN, which
// turns the outputs they take part in into NaN as the unquantised product does.

#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "fp8_convert.h"
#include "operators.h"

namespace muonh {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// quantiser

template <bool NT, typename V>
__device__ __forceinline__ V load_vec(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load((const MUONH_GLOBAL V*)p);
  return ld_global<V>(p);
}

// Eight consecutive elements of a row in the type they are stored in.  Rows may
// start at any element: global loads of any width need no more than element
// alignment on gfx950.  kWords registers hold them; for bf16 a magnitude is 15
// bits and two of them share a register.
template <typename T> struct Row8;
template <> struct Row8<uint16_t> {
  static constexpr int kWords = 4;
  static constexpr uint32_t kInf = 0x7f80u;      // magnitudes from here on are Inf or NaN
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  uint32_t w[kWords];
  template <bool NT>
  __device__ __forceinline__ void load(const uint16_t* p) {
    const vec r = load_vec<NT, vec>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = r[k];
  }
  __device__ __forceinline__ void set(int j, const uint16_t* p) {
    w[j >> 1] |= (uint32_t)ld_global<uint16_t>(p) << (16 * (j & 1));
  }
  __device__ __forceinline__ float value(int j) const {
    return __uint_as_float((j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t magnitude(int k) const { return w[k] & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
  }
  // The larger half, and a magnitude as fp32 bits.
  static __device__ __forceinline__ uint32_t fold(uint32_t m) { return max(m & 0xffffu, m >> 16); }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m << 16; }
  static __device__ __forceinline__ uint32_t column(const uint32_t (&m)[kWords], int j) {
    return (j & 1) ? m[j >> 1] >> 16 : m[j >> 1] & 0xffffu;
  }
  // Magnitudes with Inf and NaN taken as zero.
  static __device__ __forceinline__ uint32_t finite(uint32_t m) {
    const uint32_t lo = m & 0xffffu, hi = m >> 16;
    return (lo < kInf ? lo : 0u) | ((hi < kInf ? hi : 0u) << 16);
  }
};
template <> struct Row8<float> {
  static constexpr int kWords = 8;
  static constexpr uint32_t kInf = 0x7f800000u;
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(4)));
  uint32_t w[kWords];
  template <bool NT>
  __device__ __forceinline__ void load(const float* p) {
    const vec lo = load_vec<NT, vec>(p), hi = load_vec<NT, vec>(p + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = lo[k];
      w[4 + k] = hi[k];
    }
  }
  __device__ __forceinline__ void set(int j, const float* p) { w[j] = __float_as_uint(ld_global<float>(p)); }
  __device__ __forceinline__ float value(int j) const { return __uint_as_float(w[j]); }
  __device__ __forceinline__ uint32_t magnitude(int k) const { return w[k] & 0x7fffffffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t fold(uint32_t m) { return m; }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
  static __device__ __forceinline__ uint32_t column(const uint32_t (&m)[kWords], int j) { return m[j]; }
  static __device__ __forceinline__ uint32_t finite(uint32_t m) { return m < kInf ? m : 0u; }
};

// Four consecutive elements of a row, and column j of four rows.
__device__ __forceinline__ uint32_t quantize_row4(const Row8<uint16_t>& v, int h, float scale) {
  return quantize4(v.w[2 * h], v.w[2 * h + 1], scale);
}
__device__ __forceinline__ uint32_t quantize_row4(const Row8<float>& v, int h, float scale) {
  return quantize4(v.value(4 * h), v.value(4 * h + 1), v.value(4 * h + 2), v.value(4 * h + 3), scale);
}
__device__ __forceinline__ uint32_t quantize_col4(const Row8<uint16_t> (&v)[4], int j, float scale) {
  const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
  return quantize4(__builtin_amdgcn_perm(v[1].w[j >> 1], v[0].w[j >> 1], sel),
                   __builtin_amdgcn_perm(v[3].w[j >> 1], v[2].w[j >> 1], sel), scale);
}
__device__ __forceinline__ uint32_t quantize_col4(const Row8<float> (&v)[4], int j, float scale) {
  return quantize4(v[0].value(j), v[1].value(j), v[2].value(j), v[3].value(j), scale);
}

constexpr int kQuantThreads = kQuantizeThreads;
constexpr int kQuantWaves = kQuantThreads / 64;
constexpr int kQuantRows = kFp8Tile * kFp8Tile / kQuantThreads / 8;   // rows per thread
static_assert(kQuantRows == 4, "a thread's rows fill one 4-byte unit of the column form");

// LDS of one tile.  Column form: row c is column c of x, 32 units of 4 rows;
// unit u of row c sits at u ^ (2 ((c >> 3) & 15)), so that one store's 16 columns
// (8 apart) and 4 units meet each bank twice, the least for 64 lanes.
template <typename T>
struct QuantLds {
  __attribute__((aligned(16))) uint8_t tile[kFp8Tile * kFp8Tile];
  __attribute__((aligned(16))) uint32_t colmax[kQuantWaves][16 * Row8<T>::kWords];
};

// Quantises and writes the tile (tr, tc) that a workgroup holds: thread t has
// columns 8 (t % 16) .. + 7 of rows 4 (t / 16) .. + 3 in v, zeros behind the
// matrix.  A 16-lane row thus covers a row's group of 128 and a thread holds 4
// consecutive values of each of its columns: the row form leaves as 8 bytes per
// row, the column form goes through LDS as one 4-byte unit per column.  The
// padding up to a multiple of 128 is written as zeros.
//
// Bound by HBM (one read, one write per form): 8192 x 2048 bf16 to both forms
// takes 15 us (4.5 TB/s).  What a thread does per element is kept to a mask, two
// packed maxima and a conversion per form that scales as it converts; Inf and
// NaN take a path of their own, per thread.
template <typename T, bool SQUARE>
__device__ __forceinline__ void write_forms(const Row8<T> (&v)[4], const QuantArgs& p, uint32_t tr, uint32_t tc,
                                            QuantLds<T>& lds) {
  typedef Row8<T> Row;
  constexpr int W = Row::kWords;
  auto& tile = lds.tile;
  auto& colmax = lds.colmax;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t r0 = (int64_t)tr * kFp8Tile + rg * 4, c0 = (int64_t)tc * kFp8Tile + cg * 8;

  // Largest magnitudes of the thread's rows, and of its columns.
  uint32_t rowmax[4], cmax[W];
  auto maxima = [&](auto keep) {
#pragma unroll
    for (int k = 0; k < W; ++k) cmax[k] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const uint32_t a = keep(v[i].magnitude(k));
        m = Row::larger(m, a);
        cmax[k] = Row::larger(cmax[k], a);
      }
      rowmax[i] = Row::fold(m);
    }
  };
  maxima([](uint32_t m) { return m; });
  const bool special = max(max(rowmax[0], rowmax[1]), max(rowmax[2], rowmax[3])) >= Row::kInf;
  if (special) maxima([](uint32_t m) { return Row::finite(m); });

  uint32_t tile_byte = 0;
  if constexpr (SQUARE) {
    uint32_t m = max16(max(max(rowmax[0], rowmax[1]), max(rowmax[2], rowmax[3])));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if (lane == 0) colmax[wave][0] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kQuantWaves; ++w) m = max(m, colmax[w][0]);
    tile_byte = scale_byte(Row::bits(m));
  }

  if (p.q) {
    // bytes of this tile's scale column, and zeros behind the last one
    const int64_t kb = (p.cols + kFp8Block - 1) / kFp8Block;
    const int nzero = (int64_t)tc == kb - 1 ? (int)((4 - (kb & 3)) & 3) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t byte = SQUARE ? tile_byte : scale_byte(Row::bits(max16(rowmax[i])));
      if (r0 + i >= p.rows) continue;
      u32x2_t o;
      if (!special) {
        const float scale = __uint_as_float(byte << 23);
        o = u32x2_t{quantize_row4(v[i], 0, scale), quantize_row4(v[i], 1, scale)};
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          o[h] = pack_fp8(scaled(v[i].value(4 * h), byte), scaled(v[i].value(4 * h + 1), byte),
                          scaled(v[i].value(4 * h + 2), byte), scaled(v[i].value(4 * h + 3), byte));
      }
      st_global<u32x2_t>(p.q + (r0 + i) * p.ldq + c0, o);
      if (cg == 0 && (!SQUARE || (rg == 0 && i == 0))) {
        uint8_t* s = p.s + (SQUARE ? (int64_t)tr : r0 + i) * p.lds + tc;
        st_global<uint8_t>(s, (uint8_t)byte);
        for (int z = 1; z <= nzero; ++z) st_global<uint8_t>(s + z, (uint8_t)0);
      }
    }
  }

  if (p.qt) {
    if constexpr (!SQUARE) {
      // columns: over the wavefront's 4 groups of rows, then over the wavefronts
#pragma unroll
      for (int k = 0; k < W; ++k) {
        cmax[k] = Row::larger(cmax[k], (uint32_t)__shfl_xor((int)cmax[k], 16, 64));
        cmax[k] = Row::larger(cmax[k], (uint32_t)__shfl_xor((int)cmax[k], 32, 64));
      }
      if (lane < 16) {
#pragma unroll
        for (int k = 0; k < W; ++k) colmax[wave][cg * W + k] = cmax[k];
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQuantWaves; ++w)
#pragma unroll
        for (int k = 0; k < W; ++k) cmax[k] = Row::larger(cmax[k], colmax[w][cg * W + k]);
    }
    const int64_t kb = (p.rows + kFp8Block - 1) / kFp8Block;
    const int64_t cbase = (int64_t)tc * kFp8Tile;
    const int nzero = (int64_t)tr == kb - 1 ? (int)((4 - (kb & 3)) & 3) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t byte = SQUARE ? tile_byte : scale_byte(Row::bits(Row::column(cmax, j)));
      uint32_t o;
      if (!special)
        o = quantize_col4(v, j, __uint_as_float(byte << 23));
      else
        o = pack_fp8(scaled(v[0].value(j), byte), scaled(v[1].value(j), byte), scaled(v[2].value(j), byte),
                     scaled(v[3].value(j), byte));
      const int c = cg * 8 + j;   // (c >> 3) & 15 == cg
      *reinterpret_cast<uint32_t*>(&tile[c * kFp8Tile + ((rg ^ (2 * cg)) << 2)]) = o;
      if (rg == 0 && (SQUARE ? c == 0 : cbase + c < p.cols)) {
        uint8_t* s = p.st + (SQUARE ? (int64_t)tc : cbase + c) * p.ldst + tr;
        st_global<uint8_t>(s, (uint8_t)byte);
        for (int z = 1; z <= nzero; ++z) st_global<uint8_t>(s + z, (uint8_t)0);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kFp8Tile * kFp8Tile / 16 / kQuantThreads; ++k) {
      const int idx = k * kQuantThreads + tid;
      const int c = idx >> 3, ch = idx & 7, g = (c >> 3) & 15;
      if (cbase + c >= p.cols) continue;
      // units 4 ch .. + 3: chunk ch ^ (g / 2), its halves swapped where g is odd
      const u32x4_t r = *reinterpret_cast<const u32x4_t*>(&tile[c * kFp8Tile + ((ch ^ (g >> 1)) << 4)]);
      st_global<u32x4_t>(p.qt + (cbase + c) * p.ldqt + (int64_t)tr * kFp8Tile + ch * 16,
                         (g & 1) ? u32x4_t{r[2], r[3], r[0], r[1]} : r);
    }
  }
}

// Elements 4 rows x 8 columns of thread t's place in tile (tr, tc) of x.
template <bool NT, typename T>
__device__ __forceinline__ void load_tile(Row8<T> (&v)[4], const T* x, int64_t rows, int64_t cols, int64_t ldx,
                                          uint32_t tr, uint32_t tc) {
  const int64_t r0 = (int64_t)tr * kFp8Tile + (threadIdx.x >> 4) * 4;
  const int64_t c0 = (int64_t)tc * kFp8Tile + (threadIdx.x & 15) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < Row8<T>::kWords; ++k) v[i].w[k] = 0;
    if (r0 + i < rows) {
      const T* src = x + (r0 + i) * ldx + c0;
      if (c0 + 8 <= cols) {
        v[i].template load<NT>(src);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < cols) v[i].set(j, src + j);
      }
    }
  }
}

// Activations and gradients have just been written and are read here for the
// last time: non-temporal loads (a norm and the quantisation of its output,
// 8192 x 2048 bf16: 27.0 us, 28.2 with ordinary loads).  Weights have not, and
// are read again by the next step (6144 x 2048 fp32: 12.7 us with ordinary
// loads, 17.5).  The forms are stored ordinarily, as a product reads them next
// (quantisation and product, 8192 x 2048 x 6144: 116 us, 128 with non-temporal
// stores).
template <typename T, bool SQUARE>
__global__ __launch_bounds__(kQuantThreads) void block_quantize_kernel(QuantArgs p, uint32_t ctiles) {
  __shared__ QuantLds<T> lds;
  const uint32_t tr = blockIdx.x / ctiles, tc = blockIdx.x % ctiles;
  Row8<T> v[4];
  load_tile<!SQUARE, T>(v, reinterpret_cast<const T*>(p.x), p.rows, p.cols, p.ldx, tr, tc);
  write_forms<T, SQUARE>(v, p, tr, tc, lds);
}

// The forms of y = (h r) w, an RMS norm whose rows' r = 1 / rms are given: y is
// formed in fp32 as the tile is read, so it is rounded once, to E4M3, and never
// stored.  The order of the two products is norm_forward's.
template <typename T>
__global__ __launch_bounds__(kQuantThreads) void norm_quantize_kernel(QuantArgs p, const float* __restrict__ weight,
                                                                      const float* __restrict__ rstd, uint32_t ctiles) {
  __shared__ QuantLds<float> lds;
  const uint32_t tr = blockIdx.x / ctiles, tc = blockIdx.x % ctiles;
  Row8<T> h[4];
  load_tile<false, T>(h, reinterpret_cast<const T*>(p.x), p.rows, p.cols, p.ldx, tr, tc);
  const int64_t r0 = (int64_t)tr * kFp8Tile + (threadIdx.x >> 4) * 4;
  const int64_t c0 = (int64_t)tc * kFp8Tile + (threadIdx.x & 15) * 8;
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  float w[8], r[4];
  if (c0 + 8 <= p.cols) {
    const vec lo = ld_global<vec>(weight + c0), hi = ld_global<vec>(weight + c0 + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = lo[j];
      w[4 + j] = hi[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c0 + j < p.cols ? weight[c0 + j] : 0.0f;
  }
  if (r0 + 4 <= p.rows) {
    const vec a = ld_global<vec>(rstd + r0);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = a[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = r0 + i < p.rows ? rstd[r0 + i] : 0.0f;
  }
  Row8<float> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool live = r0 + i < p.rows;
    // behind the matrix 0 r w is no zero where r or w is infinite
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i].w[j] = live && c0 + j < p.cols ? __float_as_uint(h[i].value(j) * r[i] * w[j]) : 0u;
  }
  write_forms<float, false>(v, p, tr, tc, lds);
}

// The column form alone, which is all that is left where the rows' kernel wrote the row
// form.  h stays as stored and y is formed twice, for the maxima and for the values, so a
// thread needs 80 registers and three tiles share a CU; one thread per column takes the
// wavefronts' maxima.  8192 x 2048 bf16: 14.4 us (3.5 TB/s; 18.3 with y held, two tiles).
template <typename T>
__global__ __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 6 : 4) void norm_columns_kernel(QuantArgs p, const float* __restrict__ weight,
                                                                        const float* __restrict__ rstd, uint32_t ctiles) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[kFp8Tile * kFp8Tile];
  __shared__ __attribute__((aligned(16))) uint32_t colmax[kQuantWaves][kFp8Tile], bytes[kFp8Tile];
  const uint32_t tr = blockIdx.x / ctiles, tc = blockIdx.x % ctiles;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cg = tid & 15, rg = tid >> 4;
  const int64_t cbase = (int64_t)tc * kFp8Tile, r0 = (int64_t)tr * kFp8Tile + rg * 4, c0 = cbase + cg * 8;
  // Rows behind the matrix repeat its last one, which changes no maximum, and their bytes
  // are cleared at the end; columns behind it are not stored.
  Row8<T> h[4];
  float w[8], r[4];
  const bool inside = c0 + 8 <= p.cols;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = min(r0 + i, p.rows - 1);
    const T* src = reinterpret_cast<const T*>(p.x) + at * p.ldx + c0;
    r[i] = rstd[at];
    if (inside) {
      h[i].template load<false>(src);
    } else {
#pragma unroll
      for (int k = 0; k < Row8<T>::kWords; ++k) h[i].w[k] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < p.cols) h[i].set(j, src + j);
    }
  }
  if (inside) {
    typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
    const vec lo = ld_global<vec>(weight + c0), hi = ld_global<vec>(weight + c0 + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = lo[j];
      w[4 + j] = hi[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c0 + j < p.cols ? weight[c0 + j] : 0.0f;
  }
  auto y = [&](int i, int j) { return h[i].value(j) * r[i] * w[j]; };
  uint32_t cmax[8];
  bool special = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = __float_as_uint(y(i, j)) & 0x7fffffffu;
      special |= m >= 0x7f800000u;
      most = max(most, m < 0x7f800000u ? m : 0u);
    }
    // over the wavefront's four rows of 16 lanes
    const auto a = __builtin_amdgcn_permlane16_swap(most, most, false, false);
    most = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(most, most, false, false);
    cmax[j] = max((uint32_t)b[0], (uint32_t)b[1]);
  }
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      *reinterpret_cast<u32x4_t*>(&colmax[wave][cg * 8 + j]) = u32x4_t{cmax[j], cmax[j + 1], cmax[j + 2], cmax[j + 3]};
  }
  __syncthreads();
  if (tid < kFp8Tile) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < kQuantWaves; ++v) m = max(m, colmax[v][tid]);
    const uint32_t byte = scale_byte(m);
    bytes[tid] = byte;
    if (cbase + tid < p.cols) {
      const int64_t kb = (p.rows + kFp8Block - 1) / kFp8Block;
      uint8_t* s = p.st + (cbase + tid) * p.ldst + tr;
      st_global<uint8_t>(s, (uint8_t)byte);
      const int nzero = (int64_t)tr == kb - 1 ? (int)((4 - (kb & 3)) & 3) : 0;
      for (int z = 1; z <= nzero; ++z) st_global<uint8_t>(s + z, (uint8_t)0);
    }
  }
  __syncthreads();
  const int64_t live = p.rows - r0;   // of the thread's rows
  const uint32_t keep = live >= 4 ? 0xffffffffu : live <= 0 ? 0u : (1u << (8 * live)) - 1;
  // else the compiler keeps y in registers
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < Row8<T>::kWords; ++k) asm volatile("" : "+v"(h[i].w[k]));
  uint32_t* const unit = reinterpret_cast<uint32_t*>(&tile[cg * 8 * kFp8Tile + ((rg ^ (2 * cg)) << 2)]);   // QuantLds' layout
  if (special) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t byte = bytes[cg * 8 + j];
      unit[j * kFp8Tile / 4] =
          keep & pack_fp8(scaled(y(0, j), byte), scaled(y(1, j), byte), scaled(y(2, j), byte), scaled(y(3, j), byte));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      unit[j * kFp8Tile / 4] = keep & quantize4(y(0, j), y(1, j), y(2, j), y(3, j), __uint_as_float(bytes[cg * 8 + j] << 23));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kFp8Tile * kFp8Tile / 16 / kQuantThreads; ++k) {
    const int idx = k * kQuantThreads + tid;
    const int c = idx >> 3, ch = idx & 7, g = (c >> 3) & 15;
    if (cbase + c >= p.cols) continue;
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(&tile[c * kFp8Tile + ((ch ^ (g >> 1)) << 4)]);
    st_global<u32x4_t>(p.qt + (cbase + c) * p.ldqt + (int64_t)tr * kFp8Tile + ch * 16,
                       (g & 1) ? u32x4_t{q[2], q[3], q[0], q[1]} : q);
  }
}

// The update of a MuonH step, W <- k1 W - k2 u, that also writes the block-scaled
// forms of the updated W: one 128 x 128 tile of one matrix per workgroup, so W is
// read and written once and never read again for its quantisation.  The update's
// arithmetic is update_kernel's (the product k2 u rounded, then one fused
// multiply-add), so W comes out bitwise the same.  Bound by HBM: 12 bytes per
// parameter at 5.5 TB/s over 1.41 G parameters (3.08 ms; the plain update takes
// 2.16 ms and a separate quantisation 2.4 more).
template <typename U>
__global__ __launch_bounds__(kQuantThreads) void update_quantize_kernel(
    const StepTile* __restrict__ tiles, const QuantArgs* __restrict__ outs, const MatGeom* __restrict__ geo,
    const MatPtrs* __restrict__ ptrs, const MatScalars* __restrict__ scal) {
  __shared__ QuantLds<float> lds;
  const StepTile t = tiles[blockIdx.x];
  const QuantArgs p = outs[t.mat];
  const int64_t rows = p.rows, cols = p.cols;
  float* w = ptrs[t.mat].w;
  const float k1 = scal[t.mat].k1, k2 = scal[t.mat].k2;
  Row8<float> v[4];
  Row8<U> u[4];
  load_tile<true, float>(v, w, rows, cols, cols, t.tr, t.tc);
  load_tile<true, U>(u, reinterpret_cast<const U*>(geo[t.mat].U), rows, cols, cols, t.tr, t.tc);
  const int64_t r0 = (int64_t)t.tr * kFp8Tile + (threadIdx.x >> 4) * 4;
  const int64_t c0 = (int64_t)t.tc * kFp8Tile + (threadIdx.x & 15) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[i].w[j] = __float_as_uint(__builtin_fmaf(k1, v[i].value(j), -(k2 * u[i].value(j))));
    if (r0 + i < rows) {
      float* dst = w + (r0 + i) * cols + c0;
      if (c0 + 8 <= cols) {
        typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __builtin_nontemporal_store(vec{v[i].w[4 * h], v[i].w[4 * h + 1], v[i].w[4 * h + 2], v[i].w[4 * h + 3]},
                                      (MUONH_GLOBAL vec*)(dst + 4 * h));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (c0 + j < cols) st_global<float>(dst + j, v[i].value(j));
          else v[i].w[j] = 0;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i].w[j] = 0;   // k1 * 0 may be NaN where the step is
    }
  }
  write_forms<float, true>(v, p, t.tr, t.tc, lds);
}

// ---------------------------------------------------------------------------
// product
//
// Two arithmetics, chosen by the output's type.  The FP8 matrix unit adds the
// products of 8 consecutive k after aligning them to the largest, keeping 14
// bits: at most 7 2^-13 of S = sum |a_k b_k| is lost.  On normal operands (K from 8
// to 16384) that is 2.0e-5 of the result in the 2-norm, which bf16's own rounding
// (1.7e-3) hides: 1.5% of the results of 8192 x 12288 x 2048 round to the other
// neighbour, and the error against 64 bits is 1.6619e-3 for 1.6618e-3 with fp32
// sums.  Sums that cancel are off by 3e-7 S there, 4e-6 S for values over all of
// E4M3.  So a bf16 C is computed by the scaled FP8 instructions, which also apply
// both E8M0 scales; an fp32 C by the bf16 instructions on operands widened in
// registers with their scales (exact above 2^-126), which keep full fp32 sums
// (1e-9 and 2e-8 S) at half the rate, also for callers who round them to bf16.

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 2^(byte - 127) for the conversions (which use its exponent alone).
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 E4M3 bytes -> 8 bf16, scaled.
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi, float scale) {
  bf16x8_t r;
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    r[e] = p0[e];
    r[2 + e] = p1[e];
    r[4 + e] = p2[e];
    r[6 + e] = p3[e];
  }
  return r;
}

// Epilogue of 4 consecutive columns of one row.
template <typename C>
__device__ __forceinline__ void store_c(C* c, int left, int accumulate, const f32x4_t& v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= left) break;
    float r = v[e];
    if constexpr (sizeof(C) == 2) {
      if (accumulate) r += bf16_to_f32(ld_global<uint16_t>(c + e));
      st_global<uint16_t>(c + e, f32_to_bf16(r));
    } else {
      if (accumulate) r += ld_global<float>(c + e);
      st_global<float>(c + e, r);
    }
  }
}

// Narrow products: up to 16 rows (or columns), where reading the other operand is
// all there is to do and only many loads in flight per CU reach HBM's rate.  16 x
// 16 outputs per workgroup, its wavefronts splitting the blocks of the
// contraction.  One 16x16x128 scaled MFMA takes exactly one block of 128; every
// lane of a row carries the row's own scale byte and both operands are laid out
// alike, so the K order inside an instruction does not matter.  The operands are
// swapped (B first): lane l then holds columns 4 (l / 16) .. + 3 of row l % 16.

// multiplies 32 bytes per lane of one block into acc
template <typename C>
__device__ __forceinline__ void multiply16(f32x4_t& acc, const u32x4_t& a0, const u32x4_t& a1, const u32x4_t& b0,
                                           const u32x4_t& b1, uint32_t ea, uint32_t eb) {
  if constexpr (sizeof(C) == 2) {
    i32x8_t fa, fb;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      fa[e] = (int)a0[e];
      fa[4 + e] = (int)a1[e];
      fb[e] = (int)b0[e];
      fb[4 + e] = (int)b1[e];
    }
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, 0, 0, 0, (int)eb, 0, (int)ea);
  } else {
    const float va = scale_value(ea), vb = scale_value(eb);
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(b0[e], b0[e + 1], vb), widen8(a0[e], a0[e + 1], va),
                                                    acc, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(b1[e], b1[e + 1], vb), widen8(a1[e], a1[e + 1], va),
                                                    acc, 0, 0, 0);
  }
}

// Short contractions (and pitches beyond the other kernel's offsets): operands
// straight into registers, rows behind the end read the last one and are
// dropped.  The 64 lanes of a load lie in 16 rows, which costs the address path
// four times what whole lines do: 16 x 2048 x 16384 takes 21.7 us, 12.2 through LDS.
constexpr int kDirectWaves = 4;
template <typename C>
__global__ __launch_bounds__(64 * kDirectWaves) void block_matmul_direct_kernel(BlockMatmulArgs p, uint32_t ntiles) {
  __shared__ f32x4_t part[kDirectWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = (int)(blockIdx.x / ntiles) * 16, n0 = (int)(blockIdx.x % ntiles) * 16;
  const int m = min(m0 + (lane & 15), p.m - 1), n = min(n0 + (lane & 15), p.n - 1);
  const uint8_t* a = p.a + (int64_t)m * p.lda + (lane >> 4) * 32;
  const uint8_t* b = p.b + (int64_t)n * p.ldb + (lane >> 4) * 32;
  const uint8_t* sa = p.sa + (int64_t)(m >> p.a_shift) * p.ldsa;
  const uint8_t* sb = p.sb + (int64_t)(n >> p.b_shift) * p.ldsb;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = wave; k < p.kblocks; k += kDirectWaves) {
    const u32x4_t a0 = ld_global<u32x4_t>(a + (int64_t)k * 128), a1 = ld_global<u32x4_t>(a + (int64_t)k * 128 + 16);
    const u32x4_t b0 = ld_global<u32x4_t>(b + (int64_t)k * 128), b1 = ld_global<u32x4_t>(b + (int64_t)k * 128 + 16);
    multiply16<C>(acc, a0, a1, b0, b1, ld_global<uint8_t>(sa + k), ld_global<uint8_t>(sb + k));
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  f32x4_t s = part[0][lane];
#pragma unroll
  for (int w = 1; w < kDirectWaves; ++w) s += part[w][lane];
  const int row = m0 + (lane & 15), col = n0 + (lane >> 4) * 4;
  if (row >= p.m || col >= p.n) return;
  store_c<C>(reinterpret_cast<C*>(p.c) + (int64_t)row * p.ldc + col, p.n - col, p.accumulate, s);
}

#define MUONH_LDS __attribute__((address_space(3)))

// Workgroup barrier without a memory fence (a fence would wait for every load
// in flight); the empty asm statements keep LDS accesses on their side of it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// s_waitcnt vmcnt(VM) lgkmcnt(0): all but the last VM global accesses, and all
// LDS accesses, of this wavefront are done.
template <int VM>
__device__ __forceinline__ void wait_loads() {
  static_assert(VM >= 0 && VM < 64, "vmcnt is 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (0 << 8));
  asm volatile("" ::: "memory");
}

constexpr int kBufferConfig = 0x00020000;   // raw, unformatted buffer access
constexpr int kSgMfma = 0x008, kSgVmemRead = 0x020, kSgDsRead = 0x100;
#define MUONH_SG(mask, n) __builtin_amdgcn_sched_group_barrier((mask), (n), 0)

constexpr int kTileThreads = 256;
constexpr int kScaleBlocks = 16;   // scales staged at a time, per row
// 16-byte chunk c of a 128-byte LDS row r sits at c ^ swz128(r): the rows of a
// fragment read then differ in banks whether 8 or 16 lanes are served at once.
__device__ __forceinline__ int swz128(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// The same through LDS, in whole 128-byte lines.  A step is one block of 128 of
// the contraction: 16 rows of A and of B, loaded straight into a slot of LDS that
// only its wavefront uses (no barrier), four steps ahead.  Each wavefront has a
// contiguous share of the blocks, so the scale bytes of four steps are one load.
//
// PARTS = 2: 8 x 8 outputs, for up to 8 rows (or columns).  Row 8 h + i of a slot
// is row i of the share's h-th half, so the two diagonal 8 x 8 quarters of an
// MFMA's result are the product's two parts (the others are dropped), and twice
// as many workgroups read the other operand.
//
// Bound by HBM where that operand is large: 8 x 12288 x 16384 takes 38 us (5.3
// TB/s), 16 x 24576 x 16384 85 us (4.7); 1 x 2048 x 6144 4.8 us, most of it latency.
constexpr int kNarrowSteps = 4;
constexpr int kNarrowSlot = 2 * 16 * kFp8Block;   // 16 rows of A, 16 of B

template <typename C, int WAVES, int PARTS>
__global__ __launch_bounds__(64 * WAVES) void block_matmul_narrow_kernel(BlockMatmulArgs p, uint32_t mt,
                                                                           uint32_t nt) {
  constexpr int kTile = 16 / PARTS;
  __shared__ __attribute__((aligned(16))) uint8_t slot0[WAVES * kNarrowSlot];
  __shared__ __attribute__((aligned(16))) uint8_t slot1[WAVES * kNarrowSlot];
  __shared__ __attribute__((aligned(16))) uint8_t slot2[WAVES * kNarrowSlot];
  __shared__ __attribute__((aligned(16))) uint8_t slot3[WAVES * kNarrowSlot];
  __shared__ f32x4_t part[WAVES][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Tiles of the shorter side vary first, 8 workgroups apart: on the same XCD, so
  // the longer side's panel is in its L2.
  const uint32_t few = min(mt, nt), one = (blockIdx.x / kMaxXcd) % few;
  const uint32_t other = blockIdx.x / (kMaxXcd * few) * kMaxXcd + blockIdx.x % kMaxXcd;
  if (other >= max(mt, nt)) return;
  const int m0 = (int)(mt < nt ? one : other) * kTile, n0 = (int)(mt < nt ? other : one) * kTile;
  const int mrows = min(kTile, p.m - m0), nrows = min(kTile, p.n - n0);
  const int per = (p.kblocks + WAVES * PARTS - 1) / (WAVES * PARTS);

  // loads
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a + (int64_t)m0 * p.lda), (short)0, (int)((mrows - 1) * p.lda) + p.kblocks * kFp8Block,
      kBufferConfig);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.b + (int64_t)n0 * p.ldb), (short)0, (int)((nrows - 1) * p.ldb) + p.kblocks * kFp8Block,
      kBufferConfig);
  constexpr int kNowhere = 0x7ffffff0;   // behind every range: no memory access, zeros
  int aoff[2], boff[2], kfirst[2], kcount[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lrow = (lane >> 3) + 8 * j;              // row of the slot
    const int row = PARTS == 1 ? lrow : lane >> 3;
    const int worker = PARTS == 1 ? wave : wave * PARTS + j;
    kfirst[j] = worker * per;                          // its share of the blocks, maybe none
    kcount[j] = min(per, p.kblocks - worker * per);
    const int chunk = ((lane & 7) ^ swz128(lrow)) * 16;
    aoff[j] = row < mrows ? (int)(row * p.lda) + chunk : kNowhere;
    boff[j] = row < nrows ? (int)(row * p.ldb) + chunk : kNowhere;
  }
  auto load_step = [&](uint8_t (&slot)[WAVES * kNarrowSlot], int i) {
    MUONH_LDS uint8_t* d = (MUONH_LDS uint8_t*)slot + wave * kNarrowSlot;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = i < kcount[j];
      const int k = in ? (kfirst[j] + i) * kFp8Block : 0;
      const int ao = in ? aoff[j] : kNowhere, bo = in ? boff[j] : kNowhere;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (MUONH_LDS void*)(d + j * 1024), 16, ao, k, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (MUONH_LDS void*)(d + 2048 + j * 1024), 16, bo, k, 0, 0);
    }
  };

  // fragments and scales
  const int at = lane & (kTile - 1), part_k = (lane & 15) / kTile;
  const int m = min(m0 + at, p.m - 1), n = min(n0 + at, p.n - 1);
  const int first = (wave * PARTS + part_k) * per, count = min(per, p.kblocks - first);
  const uint8_t* sa = p.sa + (int64_t)(m >> p.a_shift) * p.ldsa;
  const uint8_t* sb = p.sb + (int64_t)(n >> p.b_shift) * p.ldsb;
  typedef uint32_t word __attribute__((aligned(1)));
  // the bytes of 4 steps, from a start that keeps the 4 inside the row; 127 (times
  // the zeros that were loaded) behind the last block
  auto load_scales = [&](const uint8_t* s, int i) {
    const int k = min(first + i, ((p.kblocks + 3) & ~3) - 4);
    return ld_global<word>(s + max(k, 0)) >> (8 * min(first + i - max(k, 0), 3));
  };
  auto scale_at = [&](uint32_t w, int i, int u) { return i < count ? (w >> (8 * u)) & 0xffu : 127u; };
  const int fswz = swz128(lane & 15);
  const int c0 = ((2 * (lane >> 4)) ^ fswz) << 4, c1 = ((2 * (lane >> 4) + 1) ^ fswz) << 4;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_t a0, a1, b0, b1;
  auto read_step = [&](uint8_t (&slot)[WAVES * kNarrowSlot]) {
    const uint8_t* d = slot + wave * kNarrowSlot + (lane & 15) * kFp8Block;
    a0 = *reinterpret_cast<const u32x4_t*>(d + c0);
    a1 = *reinterpret_cast<const u32x4_t*>(d + c1);
    b0 = *reinterpret_cast<const u32x4_t*>(d + 2048 + c0);
    b1 = *reinterpret_cast<const u32x4_t*>(d + 2048 + c1);
  };
  auto multiply = [&](uint32_t ea, uint32_t eb) { multiply16<C>(acc, a0, a1, b0, b1, ea, eb); };
  load_step(slot0, 0);
  load_step(slot1, 1);
  load_step(slot2, 2);
  load_step(slot3, 3);
  uint32_t wa = load_scales(sa, 0), wb = load_scales(sb, 0);
  int i = 0;
  auto step = [&](uint8_t (&slot)[WAVES * kNarrowSlot], int u) {
    wait_loads<4 * (kNarrowSteps - 1)>();   // this step's loads are done, the next three may not be
    read_step(slot);
    wait_loads<63>();                       // the slot has been read
    load_step(slot, i + u + kNarrowSteps);
    multiply(scale_at(wa, i + u, u), scale_at(wb, i + u, u));
  };
  for (; i + kNarrowSteps < per; i += kNarrowSteps) {
    const uint32_t na = load_scales(sa, i + kNarrowSteps), nb = load_scales(sb, i + kNarrowSteps);
    step(slot0, 0);
    step(slot1, 1);
    step(slot2, 2);
    step(slot3, 3);
    wa = na;
    wb = nb;
  }
  wait_loads<0>();
  read_step(slot0);
  multiply(scale_at(wa, i, 0), scale_at(wb, i, 0));
  read_step(slot1);
  multiply(scale_at(wa, i + 1, 1), scale_at(wb, i + 1, 1));
  read_step(slot2);
  multiply(scale_at(wa, i + 2, 2), scale_at(wb, i + 2, 2));
  read_step(slot3);
  multiply(scale_at(wa, i + 3, 3), scale_at(wb, i + 3, 3));
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  const int row = m0 + at, col = n0 + (lane >> 4) * 4;
  if (part_k != 0 || (lane >> 4) * 4 >= kTile || row >= p.m || col >= p.n) return;
  // part k's outputs are 16 / PARTS rows and columns on: k kTile lanes and k kTile / 4 groups of 16
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int w = 0; w < WAVES; ++w)
#pragma unroll
    for (int h = 0; h < PARTS; ++h) s += part[w][lane + h * 5 * kTile];
  store_c<C>(reinterpret_cast<C*>(p.c) + (int64_t)row * p.ldc + col, p.n - col, p.accumulate, s);
}

// Tile of workgroup b: the hardware deals workgroups to the 8 XCDs in turn, so
// XCD x gets a contiguous share of the tile list, and the list walks groups of
// 4 tile rows column by column: the 32 tiles that run on an XCD at a time share
// 4 panels of A and 8 of B in its L2.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t mt, uint32_t nt, uint32_t& tm, uint32_t& tn) {
  const uint32_t total = mt * nt, share = total / kMaxXcd, extra = total % kMaxXcd;
  const uint32_t x = b % kMaxXcd;
  const uint32_t idx = x * share + min(x, extra) + b / kMaxXcd;
  const uint32_t g = idx / (4 * nt), rest = idx % (4 * nt), rows = min(4u, mt - 4 * g);
  tm = 4 * g + rest % rows;
  tn = rest / rows;
}

// C tile of 64 MA x 64 NB per workgroup of 4 wavefronts (2 x 2, each MA x NB
// MFMA blocks of 32 x 32).  Blocks of 128 bytes of K, whole 128-byte lines of
// every row, go straight from global memory into one of two LDS slots; each
// slot is a variable of its own, so that the compiler makes a fragment read wait
// for the loads into its own slot only.  A block is multiplied in two halves.
// During the first the wavefront reads the second's fragments; then comes the
// block's one barrier, after which its slot is free and the next block's data
// are in the other; during the second half the next block's first fragments are
// read and the block after it is loaded.
//
// 8192 x 8192 x 8192 to bf16 takes 393 us (2796 TFLOP/s), to fp32 794 us (1385);
// without the loads the former takes 363 - 458 with the scales read per lane -
// and without the fragment reads it gains 1%, so the latency of the loads into
// LDS is what is left, and the matrix unit's own pace under load.
//
// FP8: the arithmetic (see above); C: what is stored.  With a contraction split
// over `splits` workgroups, C is float and each writes its own partial matrix.
template <bool FP8, typename C, int MA, int NB>
__global__ __launch_bounds__(kTileThreads) void block_matmul_tile_kernel(BlockMatmulArgs p, uint32_t mt,
                                                                         uint32_t nt) {
  constexpr int kTileA = 64 * MA, kTileB = 64 * NB;
  constexpr int kOperandA = kTileA * kFp8Block;
  constexpr int kSlot = kOperandA + kTileB * kFp8Block;
  __shared__ __attribute__((aligned(16))) uint8_t slot0[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t slot1[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t scales[2][(kTileA + kTileB) * kScaleBlocks];

  uint32_t tm, tn;
  tile_of(blockIdx.x % (mt * nt), mt, nt, tm, tn);
  if (p.splits > 1) {
    const int k0 = (int)(blockIdx.x / (mt * nt)) * p.split_blocks;
    p.a += (int64_t)k0 * kFp8Block;
    p.b += (int64_t)k0 * kFp8Block;
    p.sa += k0;
    p.sb += k0;
    p.c = reinterpret_cast<float*>(p.c) + (int64_t)(blockIdx.x / (mt * nt)) * p.m * p.ldc;
    p.kblocks = min(p.kblocks - k0, p.split_blocks);
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  const int row0 = (int)tm * kTileA, col0 = (int)tn * kTileB;

  f32x16_t acc[MA][NB];
#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Loads: instruction i of a wavefront fills rows 16 MA wave + 8 i .. + 7 of A
  // (NB of B); lane l lands in row l / 8, slot chunk l % 8.  Rows behind the
  // matrix and blocks behind the last are out of the descriptor's range: they
  // make no memory access and leave zeros.  The range check counts the scalar
  // offset, word by word, and does not wrap where that alone is behind the range
  // (checked on the device).  The host keeps 256 rows below 2^31 bytes.
  const uint8_t* abase = p.a + (int64_t)row0 * p.lda;
  const uint8_t* bbase = p.b + (int64_t)col0 * p.ldb;
  // to the end of the last row's last block
  const int arange = (int)((min(kTileA, p.m - row0) - 1) * p.lda) + p.kblocks * kFp8Block;
  const int brange = (int)((min(kTileB, p.n - col0) - 1) * p.ldb) + p.kblocks * kFp8Block;
  const int lrow = lane >> 3;
  int avoff[2], bvoff[2];   // even and odd i
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int chunk = (lane & 7) ^ swz128(lrow + 8 * o);
    avoff[o] = (int)((wave * MA * 16 + lrow) * p.lda) + chunk * 16;
    bvoff[o] = (int)((wave * NB * 16 + lrow) * p.ldb) + chunk * 16;
  }
  auto load_block = [&](uint8_t (&slot)[kSlot], int kb) {
    const bool in = kb < p.kblocks;
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(abase), (short)0, in ? arange : 0, kBufferConfig);
    const __amdgpu_buffer_rsrc_t rb =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(bbase), (short)0, in ? brange : 0, kBufferConfig);
    MUONH_LDS uint8_t* da = (MUONH_LDS uint8_t*)slot + wave * MA * 16 * kFp8Block;
    MUONH_LDS uint8_t* db = (MUONH_LDS uint8_t*)slot + kOperandA + wave * NB * 16 * kFp8Block;
#pragma unroll
    for (int i = 0; i < 2 * (MA > NB ? MA : NB); ++i) {
      if (i < 2 * MA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (MUONH_LDS void*)(da + i * 8 * kFp8Block), 16, avoff[i & 1],
                                                 (int)(i * 8 * p.lda) + kb * kFp8Block, 0, 0);
      if (i < 2 * NB)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (MUONH_LDS void*)(db + i * 8 * kFp8Block), 16, bvoff[i & 1],
                                                 (int)(i * 8 * p.ldb) + kb * kFp8Block, 0, 0);
    }
  };

  // Fragments: block i of A is rows 32 (MA wr + i) + l % 32; lane l holds the 32
  // bytes 32 (l / 32) .. of the half block.
  const int fswz = swz128(lane & 15);
  const int aoff = (wr * MA * 32 + (lane & 31)) * kFp8Block;
  const int boff = kOperandA + (wc * NB * 32 + (lane & 31)) * kFp8Block;
  struct Frags {
    u32x4_t a[MA][2], b[NB][2];
  };
  auto read_frags = [&](Frags& f, uint8_t (&slot)[kSlot], int half) {
#pragma unroll
    for (int i = 0; i < (MA > NB ? MA : NB); ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int chunk = ((4 * half + 2 * (lane >> 5) + h) ^ fswz) << 4;
        if (i < MA) f.a[i][h] = *reinterpret_cast<const u32x4_t*>(slot + aoff + i * 32 * kFp8Block + chunk);
        if (i < NB) f.b[i][h] = *reinterpret_cast<const u32x4_t*>(slot + boff + i * 32 * kFp8Block + chunk);
      }
  };

  // Scales: 16 blocks' bytes of every row of the tile at a time in LDS (A's
  // rows, then B's), two such chunks in turn.  (Each lane reading its own rows'
  // bytes from memory touches 32 lines per load, for every block more lines
  // than the block's data: 454 against 393 us at 8192 x 8192 x 8192.)
  auto load_scales = [&](int chunk) {
#pragma unroll
    for (int q0 = 0; q0 < MA + NB; q0 += 4) {
      const int q = q0 + wave;
      if (q >= MA + NB) break;
      const bool is_a = q < MA;
      const uint8_t* base = is_a ? p.sa : p.sb;
      const int64_t pitch = is_a ? p.ldsa : p.ldsb;
      const int shift = is_a ? p.a_shift : p.b_shift, end = (is_a ? p.m : p.n) - 1, first = is_a ? row0 : col0;
      const int s0 = first >> shift, rows = (min(first + (is_a ? kTileA : kTileB) - 1, end) >> shift) - s0;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(base + s0 * pitch), (short)0, (int)(rows * pitch) + ((p.kblocks + 3) & ~3), kBufferConfig);
      const int row = (min(first + (is_a ? q : q - MA) * 64 + lane, end) >> shift) - s0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (MUONH_LDS void*)((MUONH_LDS uint8_t*)scales[chunk & 1] + q * 64 * kScaleBlocks), 16,
          (int)(row * pitch), chunk * kScaleBlocks, 0, 0);
    }
  };
  uint32_t ea[MA], eb[NB], na[MA], nb[NB];
  auto read_scales = [&](int kb) {
    const int at = min(kb, p.kblocks - 1);
    const uint8_t* s = scales[(at / kScaleBlocks) & 1] + (at % kScaleBlocks) + (lane & 31) * kScaleBlocks;
#pragma unroll
    for (int i = 0; i < MA; ++i) na[i] = s[((wr * MA + i) * 32) * kScaleBlocks];
#pragma unroll
    for (int j = 0; j < NB; ++j) nb[j] = s[(kTileA + (wc * NB + j) * 32) * kScaleBlocks];
  };

  // Operands are swapped (B first), so a lane holds 4 consecutive columns of
  // one row per group of 4 accumulators.
  auto multiply = [&](const Frags& f) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          i32x8_t fa, fb;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fa[e] = (int)f.a[i][0][e];
            fa[4 + e] = (int)f.a[i][1][e];
            fb[e] = (int)f.b[j][0][e];
            fb[4 + e] = (int)f.b[j][1][e];
          }
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb, fa, acc[i][j], 0, 0, 0, (int)eb[j], 0,
                                                                      (int)ea[i]);
        }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x8_t wa[MA], wb[NB];
#pragma unroll
        for (int i = 0; i < MA; ++i)
          wa[i] = widen8(f.a[i][q >> 1][(q & 1) * 2], f.a[i][q >> 1][(q & 1) * 2 + 1], scale_value(ea[i]));
#pragma unroll
        for (int j = 0; j < NB; ++j)
          wb[j] = widen8(f.b[j][q >> 1][(q & 1) * 2], f.b[j][q >> 1][(q & 1) * 2 + 1], scale_value(eb[j]));
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
      }
    }
  };
  // Per MFMA so many fragment reads (and loads): all of a half's are then issued
  // in its first half, and the last read has landed by the barrier.
  constexpr int kPer = MA * NB >= 8 ? 2 : 4;
  Frags f0, f1;
  auto block = [&](uint8_t (&mine)[kSlot], uint8_t (&other)[kSlot], int kb) {
#pragma unroll
    for (int i = 0; i < MA; ++i) ea[i] = na[i];
#pragma unroll
    for (int j = 0; j < NB; ++j) eb[j] = nb[j];
    read_frags(f1, mine, 1);
    multiply(f0);
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < MA * NB; ++k) {
        MUONH_SG(kSgMfma, 1);
        MUONH_SG(kSgDsRead, kPer);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<0>();   // the next block is in its slot
    lds_barrier();     // for every wavefront, and all have read theirs
    read_scales(kb + 1);
    read_frags(f0, other, 0);
    load_block(mine, kb + 2);
    multiply(f1);
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < MA * NB; ++k) {
        MUONH_SG(kSgMfma, 1);
        MUONH_SG(kSgDsRead, kPer);
        MUONH_SG(kSgVmemRead, kPer);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  load_scales(0);
  load_block(slot0, 0);
  load_block(slot1, 1);
  wait_loads<2 * (MA + NB)>();
  lds_barrier();
  read_scales(0);
  read_frags(f0, slot0, 0);
  // Behind an odd count of blocks comes one of zeros (with the last scales).
  for (int k0 = 0; k0 < p.kblocks; k0 += kScaleBlocks) {
    // the chunk before this one has been read by every wavefront
    load_scales(k0 / kScaleBlocks + 1);
    const int k1 = min(k0 + kScaleBlocks, p.kblocks);
    for (int kb = k0; kb < k1; kb += 2) {
      block(slot0, slot1, kb);
      block(slot1, slot0, kb + 1);
    }
  }
  wait_loads<0>();   // no load into LDS is in flight past this point
  lds_barrier();

  // Epilogue: the wavefront's rows go through half a slot of its own, in passes
  // of as many rows as it holds, 16-byte chunk c of row r at c ^ (r & kMask), and
  // leave as whole rows.
  uint8_t* reg = ((wave & 2) ? slot1 : slot0) + (wave & 1) * (kSlot / 2);
  constexpr int kRowBytes = 32 * NB * (int)sizeof(C);
  constexpr int kChunks = kRowBytes / 16;   // 16-byte chunks per row
  constexpr int kBlocks = kSlot / 2 / kRowBytes / 32;
  constexpr int kPass = kBlocks >= MA ? MA : kBlocks >= 2 ? 2 : 1;   // blocks of 32 rows per pass
  constexpr int kMask = kChunks % 16 == 0 ? 15 : kChunks % 8 == 0 ? 7 : 3;
  static_assert(kBlocks >= 1 && MA % kPass == 0 && kChunks % (kMask + 1) == 0, "whole blocks per pass");
  C* c = reinterpret_cast<C*>(p.c) + (int64_t)(row0 + wr * MA * 32) * p.ldc + col0 + wc * NB * 32;
  const int rows = p.m - (row0 + wr * MA * 32), cols = p.n - (col0 + wc * NB * 32);
  if (sizeof(C) == 2 && p.accumulate) {
    // added to c before the one rounding: straight to memory
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * i + (lane & 31), col = 32 * j + 8 * g + 4 * (lane >> 5);
          const f32x16_t& v = acc[i][j];
          if (r < rows && col < cols)
            store_c<C>(c + (int64_t)r * p.ldc + col, cols - col, 1, f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]});
        }
    return;
  }
#pragma unroll
  for (int i0 = 0; i0 < MA; i0 += kPass) {
#pragma unroll
    for (int i = 0; i < kPass; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * i + (lane & 31), col = 32 * j + 8 * g + 4 * (lane >> 5);
          const f32x16_t& v = acc[i0 + i][j];
          uint8_t* d = reg + r * kRowBytes + ((((col * (int)sizeof(C)) >> 4) ^ (r & kMask)) << 4);
          if constexpr (sizeof(C) == 2)
            *reinterpret_cast<u32x2_t*>(d + (col & 4) * 2) =
                u32x2_t{pack_bf16x2(v[4 * g], v[4 * g + 1]), pack_bf16x2(v[4 * g + 2], v[4 * g + 3])};
          else
            *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
        }
#pragma unroll
    for (int k = 0; k < kPass * 32 * kChunks / 64; ++k) {
      const int idx = k * 64 + lane, lr = idx / kChunks, ch = idx % kChunks;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(reg + lr * kRowBytes + ((ch ^ (lr & kMask)) << 4));
      const int r = i0 * 32 + lr, col = ch * (16 / (int)sizeof(C));
      if (r >= rows || col >= cols) continue;
      C* d = c + (int64_t)r * p.ldc + col;
      if constexpr (sizeof(C) == 2) {
        typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
        if (col + 8 <= cols) {
          st_global<vec>(d, (vec)v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < cols) st_global<uint16_t>(d + e, (uint16_t)(v[e >> 1] >> (16 * (e & 1))));
        }
      } else {
        typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
        const f32x4_t o = __builtin_bit_cast(f32x4_t, v);
        if (col + 4 <= cols) {
          vec x = o;
          if (p.accumulate) x += ld_global<vec>(d);
          st_global<vec>(d, x);
        } else {
          store_c<float>(d, cols - col, p.accumulate, o);
        }
      }
    }
  }
}

// Adds the partial matrices of a split contraction in order, 4 elements per
// thread along the rows of the (dense) partials.
template <typename C>
__global__ __launch_bounds__(256) void block_matmul_fold_kernel(const float* __restrict__ part, int splits, int64_t m,
                                                                int64_t n, C* c, int64_t ldc, int accumulate) {
  const int64_t e0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, total = m * n;
  if (e0 >= total) return;
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  if (e0 + 4 <= total) {
    f32x4_t s = ld_global<vec>(part + e0);
    for (int k = 1; k < splits; ++k) s += (f32x4_t)ld_global<vec>(part + k * total + e0);
    int64_t row = e0 / n, col = e0 % n;
    if (col + 4 <= n) {
      store_c<C>(c + row * ldc + col, 4, accumulate, s);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        store_c<C>(c + row * ldc + col, 1, accumulate, f32x4_t{s[e], 0.0f, 0.0f, 0.0f});
        if (++col == n) {
          col = 0;
          ++row;
        }
      }
    }
  } else {
    for (int64_t e = e0; e < total; ++e) {
      float s = part[e];
      for (int k = 1; k < splits; ++k) s += part[k * total + e];
      store_c<C>(c + (e / n) * ldc + e % n, 1, accumulate, f32x4_t{s, 0.0f, 0.0f, 0.0f});
    }
  }
}

template <bool FP8, typename C>
hipError_t launch_tiles(const MatmulPlan& pl, const BlockMatmulArgs& a, hipStream_t st) {
  const uint32_t mt = (uint32_t)((a.m + 64 * pl.ma - 1) / (64 * pl.ma));
  const uint32_t nt = (uint32_t)((a.n + 64 * pl.nb - 1) / (64 * pl.nb));
  const dim3 grid(mt * nt * (uint32_t)a.splits), block(kTileThreads);
#define MUONH_TILE(MA, NB)                                                                            \
  if (pl.ma == MA && pl.nb == NB) {                                                                   \
    hipLaunchKernelGGL((block_matmul_tile_kernel<FP8, C, MA, NB>), grid, block, 0, st, a, mt, nt);    \
    return hipGetLastError();                                                                         \
  }
  MUONH_TILE(4, 4)
  MUONH_TILE(4, 3)
  MUONH_TILE(3, 4)
  MUONH_TILE(2, 2)
  MUONH_TILE(1, 1)
#undef MUONH_TILE
  return hipErrorInvalidValue;
}

template <typename C>
hipError_t matmul_for(const MatmulPlan& pl, BlockMatmulArgs a, float* workspace, hipStream_t st) {
  constexpr bool kFp8 = sizeof(C) == 2;
  a.splits = 1;
  a.split_blocks = a.kblocks;
  if (pl.ma == 0) {
    const int64_t big = ((a.m + 15) / 16) * (int64_t)((a.n + 15) / 16);
    const int32_t least = std::min(a.m, a.n);
    if (narrow_direct(a)) {
      hipLaunchKernelGGL((block_matmul_direct_kernel<C>), dim3((unsigned)big), dim3(64 * kDirectWaves), 0, st, a,
                         (unsigned)((a.n + 15) / 16));
      return hipGetLastError();
    }
    // Long contractions take more workgroups (8 x 8 outputs) or wavefronts each: 8 x
    // 6144 x 16384: 4 wavefronts 25.4 us, 8 24.6, 8 x 8 outputs 21.2; 16 x 12288 x
    // 16384: 44.2 and 41.9.  Others not (8 x 6144 x 8192: 12.7, 8 x 8 outputs 14.0; 16 x
    // 6144 x 8192: 14.3, 8 wavefronts 16.3), unless most CUs are idle (8 x 64 x 8192: 4.4
    // and 3.6).
    const bool two = least <= 8 && a.kblocks >= (big <= 64 ? 64 : 128);
    const int tile = two ? 8 : 16;
    const unsigned mt = (unsigned)((a.m + tile - 1) / tile), nt = (unsigned)((a.n + tile - 1) / tile);
    const unsigned few = std::min(mt, nt), many = (std::max(mt, nt) + kMaxXcd - 1) / kMaxXcd * kMaxXcd;
    const dim3 grid(few * many);
    if (two)
      hipLaunchKernelGGL((block_matmul_narrow_kernel<C, 4, 2>), grid, dim3(256), 0, st, a, mt, nt);
    else if (a.kblocks >= 128)
      hipLaunchKernelGGL((block_matmul_narrow_kernel<C, 8, 1>), grid, dim3(512), 0, st, a, mt, nt);
    else
      hipLaunchKernelGGL((block_matmul_narrow_kernel<C, 4, 1>), grid, dim3(256), 0, st, a, mt, nt);
    return hipGetLastError();
  }
  if (pl.splits == 1) return launch_tiles<kFp8, C>(pl, a, st);
  BlockMatmulArgs part = a;
  part.splits = pl.splits;
  part.split_blocks = pl.split_blocks;
  part.c = workspace;
  part.ldc = a.n;
  part.accumulate = 0;
  const hipError_t e = launch_tiles<kFp8, float>(pl, part, st);
  if (e != hipSuccess) return e;
  const int64_t groups = ((int64_t)a.m * a.n + 1023) / 1024;
  hipLaunchKernelGGL((block_matmul_fold_kernel<C>), dim3((unsigned)groups), dim3(256), 0, st, workspace, pl.splits,
                     (int64_t)a.m, (int64_t)a.n, reinterpret_cast<C*>(a.c), a.ldc, a.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quantize(int bf16, int square, const QuantArgs& a, hipStream_t st) {
  const int64_t rt = (a.rows + kFp8Tile - 1) / kFp8Tile, ct = (a.cols + kFp8Tile - 1) / kFp8Tile;
  const dim3 grid((unsigned)(rt * ct)), block(kQuantThreads);
  const uint32_t c = (uint32_t)ct;
  if (bf16) {
    if (square)
      hipLaunchKernelGGL((block_quantize_kernel<uint16_t, true>), grid, block, 0, st, a, c);
    else
      hipLaunchKernelGGL((block_quantize_kernel<uint16_t, false>), grid, block, 0, st, a, c);
  } else {
    if (square)
      hipLaunchKernelGGL((block_quantize_kernel<float, true>), grid, block, 0, st, a, c);
    else
      hipLaunchKernelGGL((block_quantize_kernel<float, false>), grid, block, 0, st, a, c);
  }
  return hipGetLastError();
}

hipError_t launch_norm_quantize(int bf16, const QuantArgs& a, const float* weight, const float* rstd, hipStream_t st) {
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  const uint32_t c = (uint32_t)((a.cols + kFp8Tile - 1) / kFp8Tile);
  const dim3 grid((unsigned)((a.rows + kFp8Tile - 1) / kFp8Tile) * c), block(kQuantThreads);
  if (a.q) {
    if (bf16) hipLaunchKernelGGL((norm_quantize_kernel<uint16_t>), grid, block, 0, st, a, weight, rstd, c);
    else hipLaunchKernelGGL((norm_quantize_kernel<float>), grid, block, 0, st, a, weight, rstd, c);
  } else {
    if (bf16) hipLaunchKernelGGL((norm_columns_kernel<uint16_t>), grid, block, 0, st, a, weight, rstd, c);
    else hipLaunchKernelGGL((norm_columns_kernel<float>), grid, block, 0, st, a, weight, rstd, c);
  }
  return hipGetLastError();
}

hipError_t launch_update_quantize(int bf16, const StepTile* tiles, int64_t ntiles, const QuantArgs* outs,
                                  const MatGeom* geo, const MatPtrs* ptrs, const MatScalars* scal, hipStream_t st) {
  if (ntiles <= 0) return hipSuccess;
  const dim3 grid((unsigned)ntiles), block(kQuantThreads);
  if (bf16)
    hipLaunchKernelGGL((update_quantize_kernel<uint16_t>), grid, block, 0, st, tiles, outs, geo, ptrs, scal);
  else
    hipLaunchKernelGGL((update_quantize_kernel<float>), grid, block, 0, st, tiles, outs, geo, ptrs, scal);
  return hipGetLastError();
}

hipError_t launch_block_matmul(int c_bf16, const MatmulPlan& plan, const BlockMatmulArgs& a, float* workspace,
                               hipStream_t st) {
  return c_bf16 ? matmul_for<uint16_t>(plan, a, workspace, st) : matmul_for<float>(plan, a, workspace, st);
}

}  // namespace muonh
