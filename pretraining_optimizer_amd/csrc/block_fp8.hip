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

#include "device_util.h"
#include "operators.h"

namespace muonh {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// quantiser

// Eight consecutive elements widened to fp32.  Rows may start at any element:
// global loads of any width need no more than element alignment on gfx950.
template <typename T> struct Load8;
template <> struct Load8<uint16_t> {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  static __device__ __forceinline__ void full(const uint16_t* p, float (&v)[8]) {
    const vec r = __builtin_nontemporal_load((const MUONH_GLOBAL vec*)p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(r[k] << 16);
      v[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* p) {
    return bf16_to_f32(ld_global<uint16_t>(p));
  }
};
template <> struct Load8<float> {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ void full(const float* p, float (&v)[8]) {
    const vec lo = __builtin_nontemporal_load((const MUONH_GLOBAL vec*)p);
    const vec hi = __builtin_nontemporal_load((const MUONH_GLOBAL vec*)(p + 4));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = lo[k];
      v[4 + k] = hi[k];
    }
  }
  static __device__ __forceinline__ float one(const float* p) { return ld_global<float>(p); }
};

// |v| as an integer, 0 for NaN and Inf: the order of these integers is the
// order of the magnitudes.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// The scale byte e + 127 of a block from its largest finite magnitude's bits:
// with amax = (1 + f) 2^(E - 127) and 448 = 1.75 * 2^8, e = E - 135, one more
// where 1 + f > 1.75.  Subnormal amax (E = 0) ends at the least byte.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 127;
  const int b = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u);
  return (uint32_t)max(b, 0);
}

// 2^-e from the scale byte (0 .. 247, so the result is a normal number).
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ float scaled(float v, float inv) {
  const bool finite = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
  return finite ? v * inv : __uint_as_float(0x7fc00000u);
}

// Four fp32 -> four E4M3 bytes (round to nearest even), lowest byte first.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

constexpr int kQuantThreads = 256;
constexpr int kRowsPerThread = 8;

// One 128 x 128 tile of x per workgroup.  Thread t holds columns 8 (t % 16) ..
// + 7 of the eight rows 8 (t / 16) .. + 7, so a 16-lane group covers a row's
// group of 128 and one thread holds 8 consecutive values of either axis: the
// row form leaves as 8 bytes per row, the column form goes through LDS as one
// 8-byte unit per column.  Elements behind the matrix count as zeros, and the
// row form's padding up to a multiple of 128 is written as such.
template <typename T, bool SQUARE>
__global__ __launch_bounds__(kQuantThreads) void block_quantize_kernel(QuantArgs p, uint32_t ctiles) {
  // Column form of the tile: row c is column c of x, 16 units of 8 rows; unit u
  // of row c sits at u ^ ((c >> 3) & 15), which spreads one store's 16 columns
  // (8 apart) over the banks.
  __shared__ __attribute__((aligned(16))) uint8_t tile[kFp8Tile * kFp8Tile];
  __shared__ uint32_t colmax[4][kFp8Tile];

  const uint32_t tr = blockIdx.x / ctiles, tc = blockIdx.x % ctiles;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t r0 = (int64_t)tr * kFp8Tile + rg * 8, c0 = (int64_t)tc * kFp8Tile + cg * 8;
  const T* x = reinterpret_cast<const T*>(p.x);

  float v[kRowsPerThread][8];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r0 + i < p.rows) {
      const T* src = x + (r0 + i) * p.ldx + c0;
      if (c0 + 8 <= p.cols) {
        Load8<T>::full(src, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < p.cols) v[i][j] = Load8<T>::one(src + j);
      }
    }
  }

  uint32_t rowmax[kRowsPerThread], cmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    rowmax[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = finite_bits(v[i][j]);
      rowmax[i] = max(rowmax[i], u);
      cmax[j] = max(cmax[j], u);
    }
  }
  uint32_t tile_byte = 0;
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) m = max(m, rowmax[i]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if (lane == 0) colmax[0][wave] = m;
    __syncthreads();
    m = max(max(colmax[0][0], colmax[0][1]), max(colmax[0][2], colmax[0][3]));
    tile_byte = scale_byte(m);
  }

  if (p.q) {
    if constexpr (!SQUARE) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i)
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
          rowmax[i] = max(rowmax[i], (uint32_t)__shfl_xor((int)rowmax[i], off, 64));
    }
    // bytes of this tile's scale column, and zeros behind the last one
    const int64_t kb = (p.cols + kFp8Block - 1) / kFp8Block;
    const int nzero = (int64_t)tc == kb - 1 ? (int)((4 - (kb & 3)) & 3) : 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      if (r0 + i >= p.rows) continue;
      const uint32_t byte = SQUARE ? tile_byte : scale_byte(rowmax[i]);
      const float inv = inverse_scale(byte);
      u32x2_t o;
      o[0] = pack_fp8(scaled(v[i][0], inv), scaled(v[i][1], inv), scaled(v[i][2], inv), scaled(v[i][3], inv));
      o[1] = pack_fp8(scaled(v[i][4], inv), scaled(v[i][5], inv), scaled(v[i][6], inv), scaled(v[i][7], inv));
      st_global<u32x2_t>(p.q + (r0 + i) * p.ldq + c0, o);
      if (cg == 0 && (!SQUARE || (rg == 0 && i == 0))) {
        uint8_t* s = p.s + (SQUARE ? (int64_t)tr : r0 + i) * p.lds + tc;
        st_global<uint8_t>(s, (uint8_t)byte);
        for (int z = 1; z <= nzero; ++z) st_global<uint8_t>(s + z, (uint8_t)0);
      }
    }
  }

  if (p.qt) {
    float inv[8];
    if constexpr (SQUARE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = inverse_scale(tile_byte);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 16, 64));
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 32, 64));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) colmax[wave][cg * 8 + j] = cmax[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = cg * 8 + j;
        inv[j] = inverse_scale(scale_byte(max(max(colmax[0][c], colmax[1][c]), max(colmax[2][c], colmax[3][c]))));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x2_t o;
      o[0] = pack_fp8(scaled(v[0][j], inv[j]), scaled(v[1][j], inv[j]), scaled(v[2][j], inv[j]), scaled(v[3][j], inv[j]));
      o[1] = pack_fp8(scaled(v[4][j], inv[j]), scaled(v[5][j], inv[j]), scaled(v[6][j], inv[j]), scaled(v[7][j], inv[j]));
      const int c = cg * 8 + j;   // (c >> 3) & 15 == cg
      *reinterpret_cast<u32x2_t*>(&tile[c * kFp8Tile + ((rg ^ cg) << 3)]) = o;
    }
    const int64_t kb = (p.rows + kFp8Block - 1) / kFp8Block;
    const int64_t cbase = (int64_t)tc * kFp8Tile;
    if (tid < kFp8Tile && cbase + tid < p.cols && (!SQUARE || tid == 0)) {
      const uint32_t byte = SQUARE ? tile_byte
                                   : scale_byte(max(max(colmax[0][tid], colmax[1][tid]),
                                                    max(colmax[2][tid], colmax[3][tid])));
      uint8_t* s = p.st + (SQUARE ? (int64_t)tc : cbase + tid) * p.ldst + tr;
      st_global<uint8_t>(s, (uint8_t)byte);
      const int nzero = (int64_t)tr == kb - 1 ? (int)((4 - (kb & 3)) & 3) : 0;
      for (int z = 1; z <= nzero; ++z) st_global<uint8_t>(s + z, (uint8_t)0);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kFp8Tile * kFp8Tile / 16 / kQuantThreads; ++k) {
      const int idx = k * kQuantThreads + tid;
      const int c = idx >> 3, u = (idx & 7) * 2;
      if (cbase + c >= p.cols) continue;
      const int sw = (c >> 3) & 15;
      const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(&tile[c * kFp8Tile + ((u ^ sw) << 3)]);
      const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(&tile[c * kFp8Tile + (((u + 1) ^ sw) << 3)]);
      st_global<u32x4_t>(p.qt + (cbase + c) * p.ldqt + (int64_t)tr * kFp8Tile + u * 8,
                         u32x4_t{lo[0], lo[1], hi[0], hi[1]});
    }
  }
}

// ---------------------------------------------------------------------------
// product
//
// Two arithmetics, chosen by the output's type.  The FP8 matrix unit adds the
// products of 8 consecutive k after aligning them to the largest, keeping 14
// bits: sums come out 2.0e-5 off in the 2-norm (normal operands, K from 8 to
// 16384), which bf16's own rounding (1.7e-3) hides.  So a bf16 C is computed
// by the scaled FP8 instructions, which also apply both E8M0 scales; an fp32 C
// by the bf16 instructions on operands widened in registers with their scales
// (exact above 2^-126), which keep full fp32 sums (2e-7) at half the rate.

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
template <typename C, bool ACC>
__device__ __forceinline__ void store_c(C* c, int64_t off, int left, const f32x4_t& v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= left) break;
    float r = v[e];
    if constexpr (sizeof(C) == 2) {
      if constexpr (ACC) r += bf16_to_f32(c[off + e]);
      c[off + e] = f32_to_bf16(r);
    } else {
      if constexpr (ACC) r += c[off + e];
      c[off + e] = r;
    }
  }
}

constexpr int kThinThreads = 256;

// 16 x 16 outputs per workgroup, its four wavefronts splitting the blocks of
// the contraction.  One 16x16x128 scaled MFMA takes exactly one block of 128;
// every lane of a row carries the row's own scale byte and both operands are
// laid out alike, so the K order inside an instruction does not matter.
// The operands are swapped (B first): lane l then holds columns 4 (l / 16) ..
// + 3 of row l % 16.  Rows behind the end read the last one and are dropped.
template <typename C, bool ACC>
__global__ __launch_bounds__(kThinThreads) void block_matmul_thin_kernel(BlockMatmulArgs p, uint32_t ntiles) {
  __shared__ f32x4_t part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = (int)(blockIdx.x / ntiles) * 16, n0 = (int)(blockIdx.x % ntiles) * 16;
  const int m = min(m0 + (lane & 15), p.m - 1), n = min(n0 + (lane & 15), p.n - 1);
  const uint8_t* a = p.a + (int64_t)m * p.lda + (lane >> 4) * 32;
  const uint8_t* b = p.b + (int64_t)n * p.ldb + (lane >> 4) * 32;
  const uint8_t* sa = p.sa + (int64_t)(m >> p.a_shift) * p.ldsa;
  const uint8_t* sb = p.sb + (int64_t)(n >> p.b_shift) * p.ldsb;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = wave; k < p.kblocks; k += 4) {
    const u32x4_t a0 = ld_global<u32x4_t>(a + (int64_t)k * 128), a1 = ld_global<u32x4_t>(a + (int64_t)k * 128 + 16);
    const u32x4_t b0 = ld_global<u32x4_t>(b + (int64_t)k * 128), b1 = ld_global<u32x4_t>(b + (int64_t)k * 128 + 16);
    const uint32_t ea = ld_global<uint8_t>(sa + k), eb = ld_global<uint8_t>(sb + k);
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
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  const f32x4_t s = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  const int row = m0 + (lane & 15), col = n0 + (lane >> 4) * 4;
  if (row >= p.m || col >= p.n) return;
  store_c<C, ACC>(reinterpret_cast<C*>(p.c), (int64_t)row * p.ldc + col, p.n - col, s);
}

template <typename C>
hipError_t matmul_for(int accumulate, const BlockMatmulArgs& a, hipStream_t st) {
  const unsigned ntiles = (unsigned)((a.n + 15) / 16);
  const dim3 grid(ntiles * (unsigned)((a.m + 15) / 16));
  if (accumulate)
    hipLaunchKernelGGL((block_matmul_thin_kernel<C, true>), grid, dim3(kThinThreads), 0, st, a, ntiles);
  else
    hipLaunchKernelGGL((block_matmul_thin_kernel<C, false>), grid, dim3(kThinThreads), 0, st, a, ntiles);
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

hipError_t launch_block_matmul(int c_bf16, int accumulate, const BlockMatmulArgs& a, hipStream_t st) {
  return c_bf16 ? matmul_for<uint16_t>(accumulate, a, st) : matmul_for<float>(accumulate, a, st);
}

}  // namespace muonh
