// Causal attention over packed sequences with grouped heads, and its gradients
// (gfx950, bf16 operands, fp32 scores, softmax statistics and sums).
//
// For row i of a sequence and a head, with S_ij = c q_i.k_j over its rows j <= i:
//   lse_i = log sum_j exp S_ij,  P_ij = exp(S_ij - lse_i),  o_i = sum_j P_ij v_j
//   dP_ij = do_i.v_j,  delta_i = do_i.o_i,  dS_ij = c P_ij (dP_ij - delta_i)
//   dq_i = sum_j dS_ij k_j,  dk_j = sum_i dS_ij q_i,  dv_j = sum_i P_ij do_i
// dk and dv are sums over the heads of a group, too.
//
// All kernels work in 32 x 32 blocks of scores on v_mfma_f32_32x32x16_bf16, whose
// result has one column per lane (l % 32) and rows 8 (r / 4) + 4 (l / 32) + r % 4 in
// its 16 registers.  The scores are computed so that the axis which the next product
// contracts lies in the registers: rounded to bf16 in pairs, registers 8 s .. 8 s + 7
// are then the B operand of step s of that product as they are, if its A operand
// takes its 16 rows in the same order.  A comes out of LDS through the transposing
// read (ds_read_b64_tr_b16: 4 consecutive rows of one column per lane), two reads
// for rows 16 s + 4 (l / 32) .. + 3 and 8 further.  So neither scores nor
// probabilities pass through LDS.
//
// Rounding to bf16: P and dS where they become matrix operands, which the matrix unit takes
// in 16 bits at the rate that this work needs (at most 2^-8 of a term, of either sign), and the
// results, once.
//
// Tiles of 64 rows go straight from memory to LDS, the next while one is used, a
// barrier per tile.  Rows behind a sequence's end and columns behind the head's width
// are out of the buffer descriptor's range and arrive as zeros, so nothing of another
// sequence or head is read.

#include "attention.h"

#include <type_traits>
#include <utility>

#include "device_util.h"

namespace muonh {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

#define MUONH_LDS __attribute__((address_space(3)))

constexpr int kThreads = kAttentionThreads;
constexpr int kTile = 64;                // rows of a tile in LDS
constexpr int kBufferConfig = 0x00020000;
constexpr int kBehind = (int)0x80000000;  // an offset behind every descriptor's range
constexpr float kLog2e = 1.4426950408889634f;

// Row r's 16-byte chunk c sits at c ^ swizzle(r).  A row is 256 (128) bytes; 16 (8)
// rows of one chunk, as an operand read has them, and 8 rows of 4 chunks, as a
// transposing read has them, then lie in different banks.
template <int DP>
__device__ __forceinline__ int swizzle(int r) {
  return DP == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

__device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

__device__ __forceinline__ f32x16_t splat(float v) {
  f32x16_t r;
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = v;
  return r;
}

// Barrier without a memory fence, and the wait for this wavefront's loads.
__device__ __forceinline__ void arrive() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((0 << 0) | (7 << 4) | (0 << 8));   // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Score register r's row within its block of 32.
__device__ __forceinline__ constexpr int block_row(int r) { return 8 * (r / 4) + r % 4; }

// Registers 8 s .. 8 s + 7 of a block as a B operand.
__device__ __forceinline__ u32x4_t operand(const f32x16_t& v, int s) {
  u32x4_t r;
#pragma unroll
  for (int w = 0; w < 4; ++w) r[w] = pack_bf16x2(v[8 * s + 2 * w], v[8 * s + 2 * w + 1]);
  return r;
}

// The larger (the sum) of lane l's and lane l ^ 32's values.
__device__ __forceinline__ float pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The rows of a tensor [tokens, heads, dim] that a workgroup reads, from one row on.
struct Rows {
  const uint16_t* base;   // of the sequence's first row, at the head
  int64_t ld;
  int len, dim;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t at(int row, int rows) const {
    const int n = min(rows, len - row);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + row * ld), (short)0,
                                             n > 0 ? (int)(((n - 1) * ld + dim) * 2) : 0, kBufferConfig);
  }
};

// A tile's loads by WAVES wavefronts: instruction i of wavefront w fills 1024 bytes of LDS.
template <int DP, int ROWS = kTile, int WAVES = 4>
struct TileLoad {
  static constexpr int kRow = DP * 2, kChunks = DP / 8, kStep = 1024 * WAVES / kRow;   // rows per round
  static_assert(ROWS % kStep == 0 && kStep % 16 == 0, "whole rounds, the swizzle the same in each");
  int voff, step;
  __device__ __forceinline__ TileLoad(int64_t ld, int dim, int wave, int lane) {
    const int row = wave * (kStep / WAVES) + lane / kChunks, chunk = (lane % kChunks) ^ swizzle<DP>(row);
    voff = chunk * 8 < dim ? (int)(row * ld * 2) + chunk * 16 : kBehind;
    step = (int)(kStep * ld * 2);
  }
  __device__ __forceinline__ void operator()(const Rows& t, int row, MUONH_LDS uint8_t* slot, int wave) const {
    const __amdgpu_buffer_rsrc_t r = t.at(row, ROWS);
#pragma unroll
    for (int i = 0; i < ROWS / kStep; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MUONH_LDS void*)(slot + (i * WAVES + wave) * 1024), 16, voff, i * step, 0, 0);
  }
};

// Operands out of a tile in LDS.  Within a row a step or a block of columns only changes
// bits of the chunk's number, so an address is one exclusive or from the lane's first.
template <int DP>
struct TileRead {
  static constexpr int kRow = DP * 2;
  int row, tr;    // byte offsets of the lane's first operand and transposing reads
  __device__ __forceinline__ explicit TileRead(int lane) {
    row = (lane & 31) * kRow + (((lane >> 5) ^ swizzle<DP>(lane & 15)) << 4);
    const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
    tr = r * kRow + (((2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) ^ swizzle<DP>(r)) << 4) + (lane & 1) * 8;
  }
  // Rows of block `sub`, columns 16 step + 8 (l / 32) .. + 7.
  __device__ __forceinline__ u32x4_t rows(MUONH_LDS uint8_t* tile, int sub, int step) const {
    return *reinterpret_cast<MUONH_LDS u32x4_t*>(tile + sub * 32 * kRow + (row ^ (step << 5)));
  }
  // Column 32 dt + l % 32 of block `sub`, rows 16 s + 4 (l / 32) .. + 3 and 8 further.
  __device__ __forceinline__ u32x4_t columns(MUONH_LDS uint8_t* tile, int sub, int s, int dt) const {
    MUONH_LDS uint8_t* t = tile + (sub * 32 + 16 * s) * kRow;
    const u32x2_t lo = __builtin_bit_cast(
        u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUONH_LDS i16x4_t*)(t + (tr ^ (dt << 6)))));
    // 8 rows further the swizzle differs in one bit
    const u32x2_t hi = __builtin_bit_cast(
        u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUONH_LDS i16x4_t*)(t + 8 * kRow + (tr ^ (dt << 6) ^ 32))));
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  }
};

// Instruction order of N pairs of a product's steps whose operands come out of LDS: reads
// stay two pairs ahead.
constexpr int kSgMfma = 0x008, kSgDsRead = 0x100;
template <int N>
__device__ __forceinline__ void order_pairs() {
  __builtin_amdgcn_sched_group_barrier(kSgDsRead, 4, 0);
#pragma unroll
  for (int i = 0; i < N - 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 2, 0);
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(kSgMfma, 4, 0);
}

// f(0), .. f(N - 1) with constants.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// The wavefront's 32 rows from `row` on as an operand held in registers: lane l has
// row l % 32, columns 16 s + 8 (l / 32) .. + 7 of step s.
template <int DP>
__device__ __forceinline__ void load_operand(u32x4_t (&f)[DP / 16], const Rows& t, int row, int lane) {
  const __amdgpu_buffer_rsrc_t r = t.at(row, 32);
  const int base = (int)((lane & 31) * t.ld * 2);
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    const int chunk = 2 * s + (lane >> 5);
    f[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                           r, chunk * 8 < t.dim ? base + chunk * 16 : kBehind, 0, 0));
  }
}

// The sequence and the place in it of a workgroup's ROWS rows: the block of the rank-th
// most work, counted in blocks seen (KEYS = false: up to its own; true: from its own on).
// Long ones first, the short ones fill the gaps at the end (gradients of packed documents of
// 8192 tokens, with item_of's order: 349 -> 294 us).  With n_b blocks in sequence b, count(h) = sum_b
// max(0, n_b - h + 1) blocks see h or more, so the rank's h is the largest with count(h) >
// rank; a lane per sequence evaluates it.  More than 64 sequences keep their order:
// blocks are numbered from cu[b] / ROWS + b on, which leaves room for the last, cut one
// (gradients of 8192 tokens in 64 random documents 111 us, in 65 of them 126; the documents above
// 265, with 57 empty sequences more 328).
//
// Ends are taken into [0, tokens], so no cu_seqlens reads or writes outside the tensors; the
// search among more than 64 needs them not to decrease.
struct Place {
  int64_t start;   // the sequence's first row
  int len, row;    // its rows, and the workgroup's first (-1: none)
};
__device__ __forceinline__ int sequence_end(const AttentionArgs& p, int b) { return min(max(p.cu[b], 0), p.tokens); }

// The sum over the wavefront.
__device__ __forceinline__ int wave_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // from lanes 1, 2, 4, 8 below in the row of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // rows 1 and 3 from lanes 15 and 47
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // rows 2 and 3 from lane 31
  return __builtin_amdgcn_readlane(v, 63);
}

template <bool KEYS, int ROWS>
__device__ __forceinline__ Place find_place(const AttentionArgs& p, int rank) {
  const int lane = threadIdx.x & 63;
  if (p.sequences > 64) {
    const int block = KEYS ? rank : p.blocks - 1 - rank;
    int lo = 0, hi = p.sequences - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sequence_end(p, mid) / ROWS + mid <= block) lo = mid;
      else hi = mid - 1;
    }
    const int s = sequence_end(p, lo), e = max(sequence_end(p, lo + 1), s);
    const int64_t row = ((int64_t)block - s / ROWS - lo) * ROWS;
    return Place{s, e - s, row < 0 || row >= e - s ? -1 : (int)row};
  }
  int s = 0, e = 0;
  if (lane < p.sequences) {
    s = sequence_end(p, lane);
    e = max(sequence_end(p, lane + 1), s);
  }
  const int n = (e - s + ROWS - 1) / ROWS;
  int h = __builtin_amdgcn_readlane(n, 0) - rank, b = 0;   // of one sequence
  if (p.sequences > 1) {
    int top = p.blocks;
    h = 0;
    while (h < top) {   // count(h) > rank, or h = 0; count(top + 1) <= rank
      const int mid = (h + top + 1) >> 1;
      if (wave_sum(max(n - mid + 1, 0)) > rank) h = mid;
      else top = mid - 1;
    }
    // the sequences with such a block, in their order
    const uint64_t have = __ballot(n >= h);
    const int skip = rank - wave_sum(max(n - h, 0));
    const uint64_t hit = __ballot(n >= h && __popcll(have & ((1ull << lane) - 1)) == skip);
    b = hit ? __builtin_ctzll(hit) : 0;
  }
  if (h < 1) return Place{0, 0, -1};
  s = __builtin_amdgcn_readlane(s, b);
  e = __builtin_amdgcn_readlane(e, b);
  return Place{s, e - s, (KEYS ? __builtin_amdgcn_readlane(n, b) - h : h - 1) * ROWS};
}

// The rows that no sequence holds, before the first and behind the last, shared out among
// the workgroups that have no rows of a sequence: zero(row, columns' first) for every 8
// columns, 16 threads a row.  With zero_rest a launch has room for one more sequence, so there
// is such a workgroup for every head.
template <bool KEYS, int ROWS, int THREADS, typename F>
__device__ __forceinline__ void each_rest(const AttentionArgs& p, int rank, F zero) {
  int first, last, share, shares;
  if (p.sequences > 64) {
    first = sequence_end(p, 0);
    last = max(sequence_end(p, p.sequences), first);
    const int used = last / ROWS + p.sequences;
    share = (KEYS ? rank : p.blocks - 1 - rank) - used;
    shares = p.blocks - used;
    if (share < 0) return;   // a number that a sequence's cut block left over
  } else {
    const int lane = threadIdx.x & 63;
    int n = 0;
    first = p.tokens;
    last = 0;
    if (lane < p.sequences) {
      first = sequence_end(p, lane);
      last = max(sequence_end(p, lane + 1), first);
      n = (last - first + ROWS - 1) / ROWS;
    }
    const int used = wave_sum(n);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      first = min(first, __shfl_xor(first, off, 64));
      last = max(last, __shfl_xor(last, off, 64));
    }
    last = max(last, first);
    share = rank - used;
    shares = p.blocks - used;
  }
  constexpr int kRowsAtOnce = THREADS / 16;
  const int64_t rest = (int64_t)first + p.tokens - last;
  for (int64_t i = (int64_t)share * kRowsAtOnce + threadIdx.x / 16; i < rest; i += (int64_t)shares * kRowsAtOnce)
    zero(i < first ? i : last - first + i, 8 * (int)(threadIdx.x % 16));
}
__device__ __forceinline__ void zero8(uint16_t* p) { st_global<u32x4_t>(p, u32x4_t{0, 0, 0, 0}); }

// Workgroup i's key head, head of its group and rank.  Workgroups i, i + 8, .. run on one
// XCD: with the key head first, an XCD's have few different ones, whose rows stay in its
// L2, and all ranks.
struct Item {
  int kv, member, rank;
};
__device__ __forceinline__ Item item_of(int kv_heads, int group) {
  const int i = blockIdx.x, rest = i / kv_heads;
  return Item{i % kv_heads, rest % group, rest / group};
}

// Where the lane's results lie: column l % 32 is a row of the tensor, registers 4 j ..
// of block dt are 4 consecutive columns of it.
__device__ __forceinline__ void store_columns(uint16_t* base, int64_t ld, int dim, int dt, const f32x16_t& acc,
                                              float factor, int lane) {
  uint16_t* out = base + (lane & 31) * ld + 4 * (lane >> 5) + 32 * dt;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (32 * dt + 8 * j < dim) {
      u32x2_t w;
      w[0] = pack_bf16x2(acc[4 * j] * factor, acc[4 * j + 1] * factor);
      w[1] = pack_bf16x2(acc[4 * j + 2] * factor, acc[4 * j + 3] * factor);
      st_global<u32x2_t>(out + 8 * j, w);
    }
}
template <int DP>
__device__ __forceinline__ void store_rows(uint16_t* base, int64_t ld, int dim, const f32x16_t (&acc)[DP / 32],
                                           float factor, int lane) {
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) store_columns(base, ld, dim, dt, acc[dt], factor, lane);
}

// One wavefront's sums in LDS: block dt, registers 4 j .. + 3 of lane l at (4 dt + j) 64 + l.
typedef MUONH_LDS f32x4_t* SumsInLds;
template <int DP>
__device__ __forceinline__ void put_sums(SumsInLds at, const f32x16_t (&sum)[DP / 32], int lane) {
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      at[(4 * dt + j) * 64 + lane] = f32x4_t{sum[dt][4 * j], sum[dt][4 * j + 1], sum[dt][4 * j + 2], sum[dt][4 * j + 3]};
}
__device__ __forceinline__ f32x16_t take_sums(SumsInLds at, int dt, int lane) {
  f32x16_t v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x4_t q = at[(4 * dt + j) * 64 + lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * j + e] = q[e];
  }
  return v;
}

// Whether any of the wavefront's values is an infinity or a NaN.
__device__ __forceinline__ bool has_special(u32x4_t v) {
  bool any = false;
#pragma unroll
  for (int w = 0; w < 4; ++w) any |= (v[w] & 0x7f80u) == 0x7f80u || (v[w] & 0x7f800000u) == 0x7f800000u;
  return any;
}

// Products of the probabilities of keys 16 h .. + 15 of the rows' own block where a value is
// an infinity or a NaN: a later row's, times its probability 0, would be a NaN.  One key at a
// time, and only the rows that see it keep the result.
template <int COLS>
__device__ __forceinline__ void add_key_by_key(f32x16_t (&acc)[COLS], const u32x4_t (&fv)[COLS], u32x4_t pr, int h, int lane) {
#pragma unroll 1
  for (int e = 0; e < 16; ++e) {
    // key 16 h + e: half (e / 4) % 2 of the lanes, word and half word
    const int word = (e >> 3) * 2 + ((e >> 1) & 1);
    const uint32_t keep = ((e >> 2) & 1) != (lane >> 5) ? 0u : (e & 1) ? 0xffff0000u : 0xffffu;
    u32x4_t mask;
#pragma unroll
    for (int w = 0; w < 4; ++w) mask[w] = w == word ? keep : 0u;
#pragma unroll
    for (int dt = 0; dt < COLS; ++dt) {
      const f32x16_t more = mfma(fv[dt] & mask, pr & mask, acc[dt]);
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[dt][r] = (lane & 31) >= 16 * h + e ? more[r] : acc[dt][r];
    }
  }
}

// The exponents of a row count from a rounded product, c times its largest score.  The
// rounding is an error of them all alike, which falls out of the result while it is small:
// at most 1 up to kFar, but 2^100 where the lowest number, as a mask, is the largest score.
// So maxima begin at -kFar, which leaves out whatever lies far below (and -inf, which minus
// itself would be a NaN), and rows whose largest score is not in between are computed again.
constexpr float kFar = 16777216.0f, kLowest = -3.4028235e38f;
__device__ __forceinline__ bool is_far(float top, float sum) {
  return top > kFar || (top <= -kFar && sum == sum);   // a NaN is the row's result already
}

// The wavefront's 32 rows again, keys and values straight from memory: the largest score is
// subtracted before the product with c, an instruction more per score, which would cost the
// main loop 4 to 6%.  Only far rows keep the result.  2 x 4096 tokens, 16/8 heads of 128, all
// rows far: 608 us; 1000 + 777 tokens, 12 heads of 64, the first 64 keys masked: 18.7 (16.3 without).
template <int DP>
__device__ __forceinline__ void far_rows(const AttentionArgs& p, const Rows& q, const Rows& k, const Rows& v, const Place& at,
                                         int row, bool far, int head, int lane) {
  constexpr int kCols = DP / 32;
  if (!__any(far)) return;
  const float c = p.scale * kLog2e;
  u32x4_t fq[DP / 16], fk[DP / 16];
  load_operand<DP>(fq, q, row, lane);
  f32x16_t acc[kCols];
#pragma unroll
  for (int dt = 0; dt < kCols; ++dt) acc[dt] = splat(0.0f);
  float top = kLowest, sum = 0.0f;
#pragma unroll 1
  for (int first = 0; first <= row; first += 32) {
    load_operand<DP>(fk, k, first, lane);
    f32x16_t s = splat(0.0f);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) s = mfma(fk[d], fq[d], s);
    float m = top;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (first == row && block_row(r) + 4 * (lane >> 5) > (lane & 31)) s[r] = -INFINITY;
      m = fmaxf(m, s[r]);
    }
    m = pair_max(m);
    const float f = __builtin_amdgcn_exp2f((top - m) * c);
    top = m;
    sum *= f;
#pragma unroll
    for (int dt = 0; dt < kCols; ++dt)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[dt][r] *= f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f((s[r] - top) * c);
      sum += s[r];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // as TileRead::columns; rows behind the end and columns behind the width are never kept
      u32x4_t fv[kCols];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int key = min(first + 16 * h + 4 * (lane >> 5) + w % 4 + 8 * (w / 4), at.len - 1);
#pragma unroll
        for (int dt = 0; dt < kCols; ++dt) {
          const uint32_t one = ld_global<uint16_t>(v.base + key * v.ld + min(32 * dt + (lane & 31), p.dim - 1));
          fv[dt][w / 2] = w % 2 ? fv[dt][w / 2] | one << 16 : one;
        }
      }
      const u32x4_t pr = operand(s, h);
      if (first == row) {
        add_key_by_key(acc, fv, pr, h, lane);
      } else {
#pragma unroll
        for (int dt = 0; dt < kCols; ++dt) acc[dt] = mfma(fv[dt], pr, acc[dt]);
      }
    }
  }
  sum = pair_sum(sum);
  if (!far) return;
  const int64_t t = at.start + row;
  store_rows<DP>(p.out + t * p.ldo + head * p.dim, p.ldo, p.dim, acc, 1.0f / sum, lane);
  if (lane < 32)
    p.lse[head * (int64_t)p.tokens + t + lane] = __builtin_fmaf(top, p.scale, __builtin_amdgcn_logf(sum) * (1.0f / kLog2e));
}

// Forward.  A wavefront holds 32 rows of q and their output transposed (a row per
// lane), and passes over the keys once with a running maximum and sum.  The output is
// rescaled only where a maximum has grown by more than 2^8 since the last time: until
// then the probabilities are up to 2^8 too large, which neither bf16 nor fp32 minds.
//
// A workgroup's tiles before its own rows are seen whole, in a loop without branches.
// Heads up to 64 columns leave room for tiles of 128 keys, whose products cover more of the
// next one's latency: 1000 + 777 tokens, 12 heads of 64, 17.8 -> 15.7 us in one part (the
// gradients do not gain by it: dq 19.7, key gradients 17.9 -> 19.5).
// 2 x 4096 tokens, 16/8 heads of 128: 147 to 177 us as the card's clock allows (935 to 775
// TFLOP/s; a large library product 1209).  Matrix unit and exponentials bind alike: a tile's
// 32 products take 1030 cycles of a SIMD, its exponentials, maxima and packing about
// 900 issue cycles of each of its two wavefronts, which overlap them only in part.  Without
// loads from memory 135 us of 154, without exponentials 135.
//
// PARTS > 1: a workgroup has 128 / PARTS rows, and PARTS wavefronts share 32 of them and
// take every PARTS-th block of 32 keys each; their sums are joined in LDS.  The chain of one
// wavefront is that much shorter, for as many times the loads: for problems of few
// workgroups (row_parts()).
template <int DP, int PARTS>
__global__ __launch_bounds__(kThreads, PARTS == 4 ? 1 : 2) void attention_forward_kernel(AttentionArgs p) {
  constexpr bool SPLIT = PARTS > 1;
  constexpr int kRows = kAttentionRows / PARTS, kKeys = SPLIT || DP == 64 ? 2 * kTile : kTile, kBytes = kKeys * DP * 2, kCols = DP / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[2 * kBytes], lds1[2 * kBytes];
  MUONH_LDS uint8_t *const slot0 = (MUONH_LDS uint8_t*)lds0, *const slot1 = (MUONH_LDS uint8_t*)lds1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = p.heads / p.kv_heads;
  const Item item = item_of(p.kv_heads, group);
  const int kv = item.kv, head = kv * group + item.member;
  const Place at = find_place<false, kRows>(p, item.rank);
  if (at.row < 0) {
    if (p.zero_rest)
      each_rest<false, kRows, kThreads>(p, item.rank, [&](int64_t t, int c) {
        if ((p.zero_rest & MUONH_ZERO_OUT) && c < p.dim) zero8(p.out + t * p.ldo + head * p.dim + c);
        if ((p.zero_rest & MUONH_ZERO_LSE) && c == 0) p.lse[head * (int64_t)p.tokens + t] = 0.0f;
      });
    return;
  }

  const Rows q{p.q + at.start * p.ldq + head * p.dim, p.ldq, at.len, p.dim};
  const Rows k{p.k + at.start * p.ldk + kv * p.dim, p.ldk, at.len, p.dim};
  const Rows v{p.v + at.start * p.ldv + kv * p.dim, p.ldv, at.len, p.dim};
  const int part = wave % PARTS, row = at.row + 32 * (wave / PARTS);   // the wavefront's share of the keys, its first row
  const int tiles = (min(at.len, at.row + kRows) + kKeys - 1) / kKeys;
  const TileLoad<DP, kKeys> load_k(p.ldk, p.dim, wave, lane), load_v(p.ldv, p.dim, wave, lane);
  const TileRead<DP> read(lane);
  load_k(k, 0, slot0, wave);
  load_v(v, 0, slot0 + kBytes, wave);
  u32x4_t fq[DP / 16];
  load_operand<DP>(fq, q, row, lane);

  f32x16_t acc[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = splat(0.0f);
  float top = -kFar, sum = 0.0f;   // both times c log2 e; the sum is of this lane's keys
  const float c = p.scale * kLog2e;

  // N blocks of 32 keys; DIAG: the last is the rows' own.
  auto step = [&](MUONH_LDS uint8_t* tile, auto n, auto diag) __attribute__((always_inline)) {
    constexpr int N = decltype(n)::value;
    constexpr bool DIAG = decltype(diag)::value;
    f32x16_t s[N];
#pragma unroll
    for (int b = 0; b < N; ++b) s[b] = splat(0.0f);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
#pragma unroll
      for (int b = 0; b < N; ++b) s[b] = mfma(read.rows(tile, b, d), fq[d], s[b]);
    if constexpr (N == 2) order_pairs<DP / 16>();
    if constexpr (DIAG) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (block_row(r) + 4 * (lane >> 5) > (lane & 31)) s[N - 1][r] = -INFINITY;
    }
    float m = s[0][0];
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, s[b][r]);
    m = pair_max(m) * c;
    if (__any(m > top + 8.0f)) {
      const float grown = fmaxf(top, m), f = __builtin_amdgcn_exp2f(top - grown);
      top = grown;
      sum *= f;
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[dt][r] *= f;
    }
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r], c, -top));
        sum += s[b][r];
      }
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_t pr = operand(s[b], h);
        u32x4_t fv[DP / 32];
        bool special = false;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) {
          fv[dt] = read.columns(tile + kBytes, b, h, dt);
          if (DIAG && b == N - 1) special |= has_special(fv[dt]);
        }
        if (DIAG && b == N - 1 && __any(special)) {
          add_key_by_key(acc, fv, pr, h, lane);
        } else {
#pragma unroll
          for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(fv[dt], pr, acc[dt]);
        }
      }
  };
  auto fetch = [&](MUONH_LDS uint8_t* tile, int j) __attribute__((always_inline)) {
    if (j < tiles) {
      load_k(k, j * kKeys, tile, wave);
      load_v(v, j * kKeys, tile + kBytes, wave);
    }
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  if constexpr (SPLIT) {
    __shared__ float stats[2][4][64];
    auto use = [&](MUONH_LDS uint8_t* tile, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 4 / PARTS; ++b) {
        const int block = PARTS * b + part, own = row / 32 - 4 * j;
        MUONH_LDS uint8_t* const mine = tile + block * 32 * DP * 2;
        if (block < own) step(mine, one, std::false_type{});
        else if (block == own) step(mine, one, std::true_type{});
      }
    };
    for (int j = 0; j < tiles; j += 2) {
      arrive();   // the tile is there, and every wavefront has read the other
      fetch(slot1, j + 1);
      use(slot0, j);
      if (j + 1 >= tiles) break;
      arrive();
      fetch(slot0, j + 2);
      use(slot1, j + 1);
    }
    stats[0][wave][lane] = top;
    stats[1][wave][lane] = pair_sum(sum);
    arrive();   // all are done with the slots, which take the sums
    auto place = [&](int w) { return (SumsInLds)(w & 1 ? slot1 : slot0) + (w >> 1) * kCols * 4 * 64; };
    static_assert(2 * kCols * 4 * 64 * 16 <= 2 * kBytes, "two wavefronts' sums fill a slot");
    put_sums<DP>(place(wave), acc, lane);
    arrive();
    const int first = wave - part;   // of the wavefronts that share the rows
    float most = stats[0][first][lane], total = 0.0f, factor[PARTS];
#pragma unroll
    for (int w = 1; w < PARTS; ++w) most = fmaxf(most, stats[0][first + w][lane]);
#pragma unroll
    for (int w = 0; w < PARTS; ++w) {
      factor[w] = __builtin_amdgcn_exp2f(stats[0][first + w][lane] - most);   // 0 of a wavefront without keys
      total += factor[w] * stats[1][first + w][lane];
    }
    const bool live = row + (lane & 31) < at.len, far = live && is_far(most, total);
    const int64_t t = at.start + row;
    if (live && !far) {
      for (int dt = part; dt < kCols; dt += PARTS) {   // the columns over the wavefronts
        f32x16_t v = splat(0.0f);
#pragma unroll
        for (int w = 0; w < PARTS; ++w) {
          const f32x16_t o = take_sums(place(first + w), dt, lane);
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] += factor[w] * o[r];
        }
        store_columns(p.out + t * p.ldo + head * p.dim, p.ldo, p.dim, dt, v, 1.0f / total, lane);
      }
      if (part == 0 && lane < 32)
        p.lse[head * (int64_t)p.tokens + t + lane] = (most + __builtin_amdgcn_logf(total)) * (1.0f / kLog2e);
    }
    if (part == 0) far_rows<DP>(p, q, k, v, at, row, far, head, lane);
    return;
  }
  // The tiles before the workgroup's rows are seen whole by all of them.
  auto full = [&](MUONH_LDS uint8_t* tile) __attribute__((always_inline)) {
    step(tile, two, std::false_type{});
    if constexpr (kKeys > kTile) step(tile + kTile * DP * 2, two, std::false_type{});
  };
  // 64 of the workgroup's own keys, the first or the second.
  auto own = [&](MUONH_LDS uint8_t* tile, int half) __attribute__((always_inline)) {
    if (wave == 2 * half) step(tile, one, std::true_type{});
    else if (wave == 2 * half + 1) step(tile, two, std::true_type{});
    else if (half == 0) step(tile, two, std::false_type{});
  };
  const int whole = at.row / kKeys;
  for (int j = 0; j + 1 < whole; j += 2) {
    arrive();   // the tile is there, and every wavefront has read the other
    fetch(slot1, j + 1);
    full(slot0);
    arrive();
    fetch(slot0, j + 2);
    full(slot1);
  }
  arrive();
  if constexpr (kKeys == kTile) {   // an even number of whole ones
    fetch(slot1, whole + 1);
    own(slot0, 0);
    if (whole + 1 < tiles) {
      arrive();
      own(slot1, 1);
    }
  } else {
    if (whole & 1) {
      fetch(slot1, whole);
      full(slot0);
      arrive();
    }
    MUONH_LDS uint8_t* const last = whole & 1 ? slot1 : slot0;
    own(last, 0);
    own(last + kTile * DP * 2, 1);
  }

  sum = pair_sum(sum);
  const bool live = row + (lane & 31) < at.len, far = live && is_far(top, sum);
  const int64_t t = at.start + row;
  if (live && !far) {
    store_rows<DP>(p.out + t * p.ldo + head * p.dim, p.ldo, p.dim, acc, 1.0f / sum, lane);
    if (lane < 32) p.lse[head * (int64_t)p.tokens + t + lane] = (top + __builtin_amdgcn_logf(sum)) * (1.0f / kLog2e);
  }
  far_rows<DP>(p, q, k, v, at, row, far, head, lane);
}

// Gradient of q, row by row as in the forward pass: S and dP from k and v, dq from dS and k.
// It also leaves what the other kernel needs of each row: -lse log2 e and -delta.
// Packed documents of 8192 tokens, 16/8 heads of 128: 117 us, three products of five (855
// TFLOP/s); 1000 + 777 tokens, 12 heads of 64: 17 us in two parts, 19 in one, bound by the longest
// workgroup's chain of tiles.
template <int DP, int PARTS>
__global__ __launch_bounds__(kThreads, PARTS == 4 ? 1 : 2) void attention_dq_kernel(AttentionGradArgs g) {
  const AttentionArgs& p = g.a;
  constexpr bool SPLIT = PARTS > 1;
  constexpr int kRows = kAttentionRows / PARTS, kKeys = SPLIT ? 2 * kTile : kTile, kBytes = kKeys * DP * 2, kCols = DP / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[2 * kBytes], lds1[2 * kBytes];
  MUONH_LDS uint8_t *const slot0 = (MUONH_LDS uint8_t*)lds0, *const slot1 = (MUONH_LDS uint8_t*)lds1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = p.heads / p.kv_heads;
  const Item item = item_of(p.kv_heads, group);
  const int kv = item.kv, head = kv * group + item.member;
  const Place at = find_place<false, kRows>(p, item.rank);
  if (at.row < 0) return;   // the other kernel clears dq's rows that no sequence holds, too

  const Rows q{p.q + at.start * p.ldq + head * p.dim, p.ldq, at.len, p.dim};
  const Rows k{p.k + at.start * p.ldk + kv * p.dim, p.ldk, at.len, p.dim};
  const Rows v{p.v + at.start * p.ldv + kv * p.dim, p.ldv, at.len, p.dim};
  const Rows o{p.out + at.start * p.ldo + head * p.dim, p.ldo, at.len, p.dim};
  const Rows d{g.dout + at.start * g.lddo + head * p.dim, g.lddo, at.len, p.dim};
  const int part = wave % PARTS, row = at.row + 32 * (wave / PARTS);
  const int tiles = (min(at.len, at.row + kRows) + kKeys - 1) / kKeys;
  const TileLoad<DP, kKeys> load_k(p.ldk, p.dim, wave, lane), load_v(p.ldv, p.dim, wave, lane);
  const TileRead<DP> read(lane);
  load_k(k, 0, slot0, wave);
  load_v(v, 0, slot0 + kBytes, wave);
  u32x4_t fq[DP / 16], fd[DP / 16];
  load_operand<DP>(fq, q, row, lane);
  load_operand<DP>(fd, d, row, lane);

  const int64_t t = head * (int64_t)p.tokens + at.start + row + (lane & 31);
  const bool live = row + (lane & 31) < at.len;
  float delta = 0.0f, lse = 0.0f;
  bool none = false;
  {
    u32x4_t fo[DP / 16];
    load_operand<DP>(fo, o, row, lane);
    if (live) lse = -p.lse[t] * kLog2e;
    // fp32 does not hold a far lse to a unit, so it says nothing of the row's probabilities,
    // and -inf is that of no key at all: both are taken as none
    none = fabsf(lse) > kFar;
    if (none) lse = -INFINITY;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        delta = __builtin_fmaf(__uint_as_float(fo[s][w] << 16), __uint_as_float(fd[s][w] << 16), delta);
        delta = __builtin_fmaf(__uint_as_float(fo[s][w] & 0xffff0000u), __uint_as_float(fd[s][w] & 0xffff0000u), delta);
      }
    delta = none ? 0.0f : -pair_sum(delta);
    if (live && lane < 32 && part == 0) {
      g.row_lse[t] = lse;
      g.row_delta[t] = delta;
    }
  }

  f32x16_t acc[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = splat(0.0f);
  const float c = p.scale * kLog2e;

  auto block = [&](MUONH_LDS uint8_t* tile, int b, auto diag) __attribute__((always_inline)) {
    f32x16_t s = splat(0.0f), ds = splat(delta);
#pragma unroll
    for (int e = 0; e < DP / 16; ++e) {
      s = mfma(read.rows(tile, b, e), fq[e], s);
      ds = mfma(read.rows(tile + kBytes, b, e), fd[e], ds);
    }
    order_pairs<DP / 16>();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      ds[r] *= __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, lse));
      if (decltype(diag)::value && block_row(r) + 4 * (lane >> 5) > (lane & 31)) ds[r] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t f = operand(ds, h);
#pragma unroll
      for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(read.columns(tile, b, h, dt), f, acc[dt]);
    }
  };
  auto fetch = [&](MUONH_LDS uint8_t* tile, int j) __attribute__((always_inline)) {
    if (j < tiles) {
      load_k(k, j * kKeys, tile, wave);
      load_v(v, j * kKeys, tile + kBytes, wave);
    }
  };
  if constexpr (SPLIT) {
    auto use = [&](MUONH_LDS uint8_t* tile, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 4 / PARTS; ++b) {
        const int mine = PARTS * b + part, own = row / 32 - 4 * j;
        if (mine < own) block(tile, mine, std::false_type{});
        else if (mine == own) block(tile, mine, std::true_type{});
      }
    };
    for (int j = 0; j < tiles; j += 2) {
      arrive();
      fetch(slot1, j + 1);
      use(slot0, j);
      if (j + 1 >= tiles) break;
      arrive();
      fetch(slot0, j + 2);
      use(slot1, j + 1);
    }
    arrive();   // all are done with the slots, which take the sums
    auto place = [&](int w) { return (SumsInLds)(w & 1 ? slot1 : slot0) + (w >> 1) * kCols * 4 * 64; };
    static_assert(2 * kCols * 4 * 64 * 16 <= 2 * kBytes, "two wavefronts' sums fill a slot");
    put_sums<DP>(place(wave), acc, lane);
    arrive();
    if (!live) return;
    const int first = wave - part;   // of the wavefronts that share the rows
    for (int dt = part; dt < kCols; dt += PARTS) {   // the columns over the wavefronts
      f32x16_t v = take_sums(place(first), dt, lane);
#pragma unroll
      for (int w = 1; w < PARTS; ++w) {
        const f32x16_t o = take_sums(place(first + w), dt, lane);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] += o[r];
      }
      store_columns(g.dq + (at.start + row) * g.lddq + head * p.dim, g.lddq, p.dim, dt, v, p.scale, lane);
    }
    return;
  }
  auto full = [&](MUONH_LDS uint8_t* tile) __attribute__((always_inline)) {
    block(tile, 0, std::false_type{});
    block(tile, 1, std::false_type{});
  };
  // as in the forward pass, an even number of whole tiles
  const int whole = at.row / kTile;
  for (int j = 0; j < whole; j += 2) {
    arrive();
    fetch(slot1, j + 1);
    full(slot0);
    arrive();
    fetch(slot0, j + 2);
    full(slot1);
  }
  arrive();
  fetch(slot1, whole + 1);
  if (wave >= 2) {
    full(slot0);
  } else {
    if (wave == 1) block(slot0, 0, std::false_type{});
    block(slot0, wave, std::true_type{});
  }
  if (whole + 1 < tiles) {
    arrive();
    if (wave == 3) block(slot1, 0, std::false_type{});
    if (wave >= 2) block(slot1, wave - 2, std::true_type{});
  }
  if (!live) return;
  store_rows<DP>(g.dq + (at.start + row) * g.lddq + head * p.dim, g.lddq, p.dim, acc, p.scale, lane);
}

// Gradients of k and v: a wavefront holds 32 rows of both and passes over the rows of
// q and dout that see them, head by head of the group.  Eight wavefronts have BLOCKS blocks
// of 32 keys: w, w + BLOCKS, .. the same, each for every PARTS-th block of rows, and their
// sums are added at the end in order.  That shortens the longest workgroup, which
// sequences of different lengths wait for (documents of 8192 tokens, 16/8 heads of 128: 4
// blocks in two parts 164 us, four wavefronts on all rows 175); problems of few
// workgroups take 2 blocks in four parts (keys_split()).
//
// Two wavefronts per SIMD, so one's products overlap the other's exponentials: a product
// takes 32 cycles and about 9 other instructions of 4 each go with it.  Of at most 256
// registers both sums take 128 and the keys 32 (D = 128), so the values' operand stays
// in LDS beside the two slots.  Operands come out of LDS two steps, or four products,
// ahead.
constexpr int kKeyThreads = 512;
template <int DP, int BLOCKS>
__global__ __launch_bounds__(kKeyThreads, 2) void attention_dkv_kernel(AttentionGradArgs g) {
  const AttentionArgs& p = g.a;
  constexpr int kWaves = kKeyThreads / 64, kParts = kWaves / BLOCKS, kKeys = 32 * BLOCKS, kRows = 32 * kParts;
  constexpr int kBytes = kRows * DP * 2, kSteps = DP / 16, kCols = DP / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[2 * kBytes], lds1[2 * kBytes], ldsv[kKeys * DP * 2];
  // -lse and -delta of a tile's rows, 64 at a time, and a place for loads of nothing
  constexpr int kRowLoads = kRows / 64, kRowValues = (kWaves > 2 * kRowLoads ? kWaves : 2 * kRowLoads) * 64;
  __shared__ __attribute__((aligned(16))) float ldsr0[kRowValues], ldsr1[kRowValues];
  MUONH_LDS uint8_t *const slot0 = (MUONH_LDS uint8_t*)lds0, *const slot1 = (MUONH_LDS uint8_t*)lds1;
  MUONH_LDS float *const rows0 = (MUONH_LDS float*)ldsr0, *const rows1 = (MUONH_LDS float*)ldsr1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key_block = wave % BLOCKS, part = wave / BLOCKS;
  const int group = p.heads / p.kv_heads;
  const Item item = item_of(p.kv_heads, 1);
  const int kv = item.kv;
  const Place at = find_place<true, kKeys>(p, item.rank);
  if (at.row < 0) {
    if (p.zero_rest)
      each_rest<true, kKeys, kKeyThreads>(p, item.rank, [&](int64_t t, int c) {
        if (c >= p.dim) return;
        if (p.zero_rest & MUONH_ZERO_DQ)
          for (int h = 0; h < group; ++h) zero8(g.dq + t * g.lddq + (kv * group + h) * p.dim + c);
        if (p.zero_rest & MUONH_ZERO_DK) zero8(g.dk + t * g.lddk + kv * p.dim + c);
        if (p.zero_rest & MUONH_ZERO_DV) zero8(g.dv + t * g.lddv + kv * p.dim + c);
      });
    return;
  }

  const Rows k{p.k + at.start * p.ldk + kv * p.dim, p.ldk, at.len, p.dim};
  const Rows v{p.v + at.start * p.ldv + kv * p.dim, p.ldv, at.len, p.dim};
  const int row = at.row + 32 * key_block;
  const TileLoad<DP, kRows, kWaves> load_q(p.ldq, p.dim, wave, lane), load_d(g.lddo, p.dim, wave, lane);
  const TileLoad<DP, kKeys, kWaves> load_v(p.ldv, p.dim, wave, lane);
  TileRead<DP> read(lane);
  // The tiles of q and dout: first those of the workgroup's own rows, head by head, then
  // the ones behind them, which see all of its keys, head by head.  Rows behind the end
  // arrive as zeros: P = exp 0, but dout, delta and q are 0.  Behind the last tile zeros are
  // loaded, from nowhere.
  const int tiles = (at.len - at.row + kRows - 1) / kRows, owns = min(tiles, (kKeys + kRows - 1) / kRows);
  const int own_trips = owns * group, trips = tiles * group;
  int lh = 0, lt = 0, lo = 0, hi = owns;   // the next to load: its head and tile, the stage's tiles
  auto fetch = [&](MUONH_LDS uint8_t* tile, MUONH_LDS float* rows) __attribute__((always_inline)) {
    const int first = at.row + lt * kRows, h = min(lh, group - 1);
    const Rows q{p.q + at.start * p.ldq + (kv * group + h) * p.dim, p.ldq, lh < group ? at.len : 0, p.dim};
    const Rows d{g.dout + at.start * g.lddo + (kv * group + h) * p.dim, g.lddo, lh < group ? at.len : 0, p.dim};
    load_q(q, first, tile, wave);
    load_d(d, first, tile + kBytes, wave);
    // wavefronts 0 .. : -lse, then as many: -delta (the others load nothing to where nobody reads)
    const int at_row = first + wave % kRowLoads * 64, rest = lh < group && wave < 2 * kRowLoads ? at.len - at_row : 0;
    const float* src = (wave < kRowLoads ? g.row_lse : g.row_delta) + (kv * group + h) * (int64_t)p.tokens + at.start + at_row;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(src), (short)0, max(min(64, rest), 0) * 4, kBufferConfig);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MUONH_LDS void*)(rows + wave * 64), 4, lane * 4, 0, 0, 0);
    const bool turn = lt + 1 == hi, second = turn && lh + 1 == group && lo == 0 && tiles > owns;
    lo = second ? owns : lo;
    hi = second ? tiles : hi;
    lh = second ? 0 : turn ? lh + 1 : lh;
    lt = turn ? lo : lt + 1;
  };
  load_v(v, at.row, (MUONH_LDS uint8_t*)ldsv, wave);
  fetch(own_trips & 1 ? slot1 : slot0, own_trips & 1 ? rows1 : rows0);
  u32x4_t fk[kSteps];
  load_operand<DP>(fk, k, row, lane);
  f32x16_t dk[kCols], dv[kCols];
#pragma unroll
  for (int dt = 0; dt < kCols; ++dt) dk[dt] = dv[dt] = splat(0.0f);
  const float c = p.scale * kLog2e;
  MUONH_LDS uint8_t* const values = (MUONH_LDS uint8_t*)ldsv + key_block * 32 * DP * 2;

  u32x4_t fp[2], fs[2];   // P and dS of a block
  // The wavefront's block of a tile: S and dP and their values.
  auto scores = [&](MUONH_LDS uint8_t* slot, MUONH_LDS float* slot_rows, bool diag) __attribute__((always_inline)) {
    MUONH_LDS uint8_t* const tile = slot + part * 32 * DP * 2;
    MUONH_LDS float* const rows = slot_rows + part * 32;
    f32x16_t s = splat(0.0f), ds = splat(0.0f);
    u32x4_t fq[2], fd[2], fv[2];
    // the addresses made from this are not worth registers over all blocks
    asm volatile("" : "+v"(read.row));
    f32x4_t lse[2], del[2];   // of two groups of four rows in turn
    auto load_values = [&](int j) __attribute__((always_inline)) {
      lse[j & 1] = *reinterpret_cast<MUONH_LDS f32x4_t*>(rows + 8 * j + 4 * (lane >> 5));
      del[j & 1] = *reinterpret_cast<MUONH_LDS f32x4_t*>(rows + kRows + 8 * j + 4 * (lane >> 5));
    };
    auto load_step = [&](auto step) __attribute__((always_inline)) {
      constexpr int e = decltype(step)::value;
      fq[e & 1] = read.rows(tile, 0, e);
      fd[e & 1] = read.rows(tile + kBytes, 0, e);
      fv[e & 1] = read.rows(values, 0, e);
    };
    load_step(std::integral_constant<int, 0>{});
    load_step(std::integral_constant<int, 1>{});
    __builtin_amdgcn_sched_barrier(0);
    each<kSteps>([&](auto step) __attribute__((always_inline)) {
      constexpr int e = decltype(step)::value;
      s = mfma(fq[e & 1], fk[e], s);
      ds = mfma(fd[e & 1], fv[e & 1], ds);
      if constexpr (e + 2 < kSteps) load_step(std::integral_constant<int, e + 2>{});
      if constexpr (e >= kSteps - 2) load_values(e - (kSteps - 2));
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, lse[r / 4 & 1][r % 4]));
      ds[r] = (ds[r] + del[r / 4 & 1][r % 4]) * s[r];
      if (r == 3 || r == 7) load_values(r / 4 + 2);
      if (diag && block_row(r) + 4 * (lane >> 5) < (lane & 31)) s[r] = ds[r] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fp[h] = operand(s, h);
      fs[h] = operand(ds, h);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Its sums.
  auto sums = [&](MUONH_LDS uint8_t* slot) __attribute__((always_inline)) {
    MUONH_LDS uint8_t* const tile = slot + part * 32 * DP * 2;
    asm volatile("" : "+v"(read.tr));
    u32x4_t ring[4];
    auto load_sum = [&](auto number) __attribute__((always_inline)) {
      constexpr int n = decltype(number)::value;
      ring[n & 3] = read.columns(n & 1 ? tile : tile + kBytes, 0, n / (2 * kCols), n / 2 % kCols);
    };
    each<4>(load_sum);
    each<4 * kCols>([&](auto number) __attribute__((always_inline)) {
      constexpr int n = decltype(number)::value, h = n / (2 * kCols), dt = n / 2 % kCols;
      if constexpr (n & 1) dk[dt] = mfma(ring[n & 3], fs[h], dk[dt]);
      else dv[dt] = mfma(ring[n & 3], fp[h], dv[dt]);
      if constexpr (n + 4 < 4 * kCols) load_sum(std::integral_constant<int, n + 4>{});
      if constexpr (n & 1) __builtin_amdgcn_sched_barrier(0);
    });
  };
  // The two wavefronts of a SIMD leave the barriers together, and would come to their
  // exponentials together: with the first half of them first, the others' products run
  // beside their exponentials and the other way round (172 -> 168 us as above).
  if (wave < 4) __builtin_amdgcn_s_setprio(1);
  // Own blocks before the keys' do not see them.  Tile t lies in slot t & 1, counted from
  // the first whole one.
#pragma unroll 1
  for (int t = -own_trips, j = 0; t < 0; ++t) {
    arrive();   // tile t is there, and all are done with the one before
    MUONH_LDS uint8_t* const slot = t & 1 ? slot1 : slot0;
    fetch(t & 1 ? slot0 : slot1, t & 1 ? rows0 : rows1);
    const int ahead = kParts * j + part - key_block;
    if (ahead >= 0) {
      scores(slot, t & 1 ? rows1 : rows0, ahead == 0);
      sums(slot);
    }
    j = j + 1 == owns ? 0 : j + 1;
  }
  for (int t = own_trips; t < trips; t += 2) {
    arrive();
    fetch(slot1, rows1);
    scores(slot0, rows0, false);
    sums(slot0);
    if (t + 1 >= trips) break;
    arrive();
    fetch(slot0, rows0);
    scores(slot1, rows1, false);
    sums(slot1);
  }
  // The parts' sums through the slots: dk, then dv.
  constexpr int kSums = kCols * 4 * 64;   // of one wavefront
  static_assert((kParts - 1) * BLOCKS * kSums * 16 <= 2 * 2 * kBytes, "all but the first part's fit the slots");
  constexpr int kInSlot = 2 * kBytes / (kSums * 16);
  auto place = [&](int i) { return (SumsInLds)(i < kInSlot ? slot0 : slot1) + i % kInSlot * kSums; };
  auto join = [&](f32x16_t (&sum)[kCols]) __attribute__((always_inline)) {
    arrive();   // all are done with what the slots held; no load into them is on its way
    if (part > 0) put_sums<DP>(place((part - 1) * BLOCKS + key_block), sum, lane);
    arrive();
    if (part == 0)
#pragma unroll
      for (int dt = 0; dt < kCols; ++dt)
#pragma unroll
        for (int o = 0; o < kParts - 1; ++o) {
          const f32x16_t more = take_sums(place(o * BLOCKS + key_block), dt, lane);
#pragma unroll
          for (int r = 0; r < 16; ++r) sum[dt][r] += more[r];
        }
  };
  join(dk);
  join(dv);
  if (part > 0 || row + (lane & 31) >= at.len) return;
  const int64_t first = at.start + row;
  store_rows<DP>(g.dk + first * g.lddk + kv * p.dim, g.lddk, p.dim, dk, p.scale, lane);
  store_rows<DP>(g.dv + first * g.lddv + kv * p.dim, g.lddv, p.dim, dv, 1.0f, lane);
}

}  // namespace

// Whether the kernels are to have smaller blocks, by n, the blocks of 128 rows x heads.
// Measured, in us of the forward pass / of the gradients (a call is 10 us at least):
//                                                  n    4 parts        2 parts        1 part
//   8000 tokens, 1 head of 128                     63   92.4 / 215                   130 / 291
//   2000 tokens, 6 heads of 128                    96   29.3 / 70.5                  38.7 / 87.7
//   4 x 300 tokens, 8 heads of 128                104   15.5 / 32.6                  12.1 / 28.9
//   1100 tokens, 12 heads of 128                  108   24.0 / 52.3                  25.1 / 56.4
//   1100 tokens, 12 heads of 64                   108   15.2 / 29.1    14.0 / 30.9   14.9 / 35.1
//   6 x 500 tokens, 4 heads of 64                 116   12.2 / 21.5    10.7 / 21.2   10.6 / 23.6
//   8000 tokens, 2 heads of 64                    126   61.1 / 125     72.4 / 141    80.5 / 175
//   4000 tokens, 4 heads of 128                   128   57.4 / 128                   69.9 / 157
//   4000 tokens, 4 heads of 64                    128   35.1 / 70.0    38.8 / 77.2   42.9 / 94.3
//   2000 tokens, 10 heads of 64                   160   29.7 / 44.3    22.3 / 47.4   23.8 / 54.2
//   500 tokens, 40 heads of 64                    160   16.8 / 29.6    10.8 / 25.7   10.7 / 26.8
//   1000 + 777 tokens, 12 heads of 64             180   22.7 / 35.9    14.7 / 33.5   15.0 / 36.2
//   1500 tokens, 16 heads of 64                   192   28.3 / 42.4    18.3 / 40.3   18.9 / 44.5
//   4 x 300 tokens, 16 heads of 64                208   16.4 / 26.5    10.8 / 22.7   10.9 / 22.0
//   700 + 50 + 900 tokens, 14 heads of 40         210   22.1 / 33.8    13.9 / 31.7   14.5 / 34.2
//   6 x 500 tokens, 8 heads of 64                 232   19.7 / 32.1    10.8 / 27.3   11.3 / 27.9
// Four parts up to a quarter of a workgroup of 128 rows per CU, long sequences up to half of
// one; two up to one of heads up to 64 columns, whose tiles of 128 keys fit a CU twice.
// n counts the entries of cu_seqlens, of empty sequences as well (the host does not see their
// lengths): 1000 tokens, 8 heads of 128, with 64 entries 24.0 / 65.0, with one 17.9 / 42.5.
//   Keys, gradients, smaller and large blocks: 1000 tokens, 8 heads of 128 (64) 42.7 and 63.7;
//   4000 tokens, 4 heads (128) 134 and 200; 1777 tokens, 12 heads of 64 (180) 38.6 and 43.2.  Worth
//   it while the large ones are less than one per CU.
static int row_parts(const AttentionArgs& a) {
  const int64_t n = attention_blocks(a.tokens, a.sequences, kAttentionRows) * a.heads;
  const bool long_ones = a.tokens >= 1024 * (int64_t)a.sequences;
  if (4 * n <= kAttentionCus || (2 * n <= kAttentionCus && long_ones)) return 4;
  return a.dim <= 64 && n < kAttentionCus ? 2 : 1;
}
static bool keys_split(const AttentionArgs& a) {
  return attention_blocks(a.tokens, a.sequences, kAttentionRows) * a.kv_heads < kAttentionCus;
}

// A kernel over blocks of `rows` rows of so many heads.
template <typename K, typename A>
static hipError_t launch_blocks(K kernel, A args, AttentionArgs& a, int rows, int heads, int threads, hipStream_t st) {
  a.blocks = (int32_t)attention_blocks(a.tokens, (int64_t)a.sequences + (a.zero_rest != 0), rows);
  hipLaunchKernelGGL(kernel, dim3((unsigned)((int64_t)a.blocks * heads)), dim3((unsigned)threads), 0, st, args());
  return hipGetLastError();
}

template <int DP>
static hipError_t forward_for(AttentionArgs& a, hipStream_t st) {
  auto args = [&] { return a; };
  const int parts = row_parts(a);
  auto kernel = parts == 4 ? attention_forward_kernel<DP, 4> : attention_forward_kernel<DP, 1>;
  if constexpr (DP == 64)
    if (parts == 2) kernel = attention_forward_kernel<DP, 2>;
  return launch_blocks(kernel, args, a, kAttentionRows / parts, a.heads, kThreads, st);
}
hipError_t launch_attention_forward(const AttentionArgs& given, hipStream_t st) {
  AttentionArgs a = given;
  return a.dim <= 64 ? forward_for<64>(a, st) : forward_for<128>(a, st);
}

template <int DP>
static hipError_t backward_for(AttentionGradArgs& g, hipStream_t st) {
  auto args = [&] { return g; };
  const int parts = row_parts(g.a);
  const bool split = keys_split(g.a);
  auto dq = parts == 4 ? attention_dq_kernel<DP, 4> : attention_dq_kernel<DP, 1>;
  if constexpr (DP == 64)
    if (parts == 2) dq = attention_dq_kernel<DP, 2>;
  const hipError_t e = launch_blocks(dq, args, g.a, kAttentionRows / parts, g.a.heads, kThreads, st);
  if (e != hipSuccess) return e;
  const auto dkv = split ? attention_dkv_kernel<DP, 2> : attention_dkv_kernel<DP, 4>;
  return launch_blocks(dkv, args, g.a, split ? 64 : kAttentionRows, g.a.kv_heads, kKeyThreads, st);
}
hipError_t launch_attention_backward(const AttentionGradArgs& given, hipStream_t st) {
  AttentionGradArgs g = given;
  return g.a.dim <= 64 ? backward_for<64>(g, st) : backward_for<128>(g, st);
}

}  // namespace muonh
