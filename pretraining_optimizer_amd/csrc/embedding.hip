// Embedding lookup with scaling, and its gradient by sorted tokens (gfx950).
//
//   out[t] = scale table[token t],  dtable[v] = scale (sum over t with token v of dout[t])
//
// A token outside the table (padding) gives zeros and adds nothing.
//
// Backward: the tokens are sorted, in a stable way, so each row's tokens stand together
// in their order of appearance; runs of 16 (or 64) sorted tokens are added by
// one group of threads each, and rows whose tokens go over a run's end are joined from
// the runs' partial sums in order.  No atomics: results are the same in every call.
// Sums are fp32, each result is rounded once.

#include "embedding.h"

#include <algorithm>

#include "row_vectors.h"

namespace muonh {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t i) {
  return wide ? ld_global<int64_t>(reinterpret_cast<const int64_t*>(tokens) + i)
              : (int64_t)ld_global<int32_t>(reinterpret_cast<const int32_t*>(tokens) + i);
}

// Groups of G threads take a token each, 8 columns per thread at a time.  Bound by HBM:
// a row is read and written once (8192 of 151936 x 2048 fp32 to bf16: 14 us, 7 TB/s, as
// frequent rows come from the cache).
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void embedding_forward_kernel(EmbeddingArgs p, int log_group) {
  const int group = 1 << log_group, t = threadIdx.x & (group - 1);
  const int64_t i = (int64_t)blockIdx.x * (kThreads >> log_group) + (threadIdx.x >> log_group);
  if (i >= p.count) return;
  const int64_t v = token_at(p.tokens, p.wide, i);
  const bool known = v >= 0 && v < p.rows;
  const T* src = reinterpret_cast<const T*>(p.table) + (known ? v : 0) * p.ldt;
  O* dst = reinterpret_cast<O*>(p.out) + i * p.ldo;
  const int cols = (int)p.cols;
  for (int c = 8 * t; c < cols; c += 8 * group) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.0f;
    if (known) {
      load8<T>(src, c, cols).widen(a);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] *= p.scale;
    }
    store8<O>(dst, c, cols, a);
  }
}

// One pass of the sort by one workgroup's keys: the stable rank of each among them.
// Thread t of wavefront w holds items 64 (N w + k) + t % 64, k < N.  Each wavefront counts its
// digits in order (equal digits of one load by a ballot per bit), and the wavefronts'
// counts are added up over the digits and, for each, over the wavefronts.
constexpr int kWaves = kSortThreads / 64;
struct SortLds {
  uint32_t count[kWaves][kSortDigits + 1];   // + 1: a digit's counters lie in different banks
};

template <int N>
__device__ __forceinline__ void count_digits(SortLds& lds, const uint32_t (&key)[N], uint32_t (&rank)[N],
                                             int64_t left, int shift, int bits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t mask = (1u << bits) - 1;
  for (int i = threadIdx.x; i < kWaves * (kSortDigits + 1); i += kSortThreads) (&lds.count[0][0])[i] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const bool live = (wave * N + k) * 64 + lane < left;
    const uint32_t d = (key[k] >> shift) & mask;
    // the lanes with this one's digit: a bit's are its ballot's or the others
    const uint64_t all = __ballot(live);
    uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
    for (int b = 0; b < bits; ++b) {
      const uint32_t bit = (uint32_t)__builtin_amdgcn_sbfe((int)d, b, 1);   // 0 or ~0
      const uint64_t m = __ballot(bit != 0);
      lo &= ~((uint32_t)m ^ bit);
      hi &= ~((uint32_t)(m >> 32) ^ bit);
    }
    const uint64_t same = (uint64_t)hi << 32 | lo;
    if (live) {
      const uint32_t before = lds.count[wave][d], at = __popcll(same & ((1ull << lane) - 1));
      rank[k] = before + at;
      // the wavefront's LDS accesses are in order: all have read before one writes
      __builtin_amdgcn_wave_barrier();
      if (at == 0) lds.count[wave][d] = before + (uint32_t)__popcll(same);
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t key_of(const EmbeddingGradArgs& p, int64_t v) {
  return v >= 0 && v < p.rows ? (uint32_t)v : (uint32_t)p.rows;
}

// Zeros in all of the table: 16 bytes per thread where the rows follow each other (one
// store each: 151936 x 2048 fp32 181 us, 6.9 TB/s; 281 us in a loop over the grid), else
// a workgroup per row.
constexpr int64_t kClearGroups = (int64_t)1 << 23;   // of one launch
template <typename O>
__global__ __launch_bounds__(kThreads) void clear_kernel(EmbeddingGradArgs p) {
  O* const table = reinterpret_cast<O*>(p.dtable);
  const int64_t n = p.rows * p.cols;
  const int64_t head = min((int64_t)((16 - (reinterpret_cast<uintptr_t>(table) & 15)) & 15) / (int64_t)sizeof(O), n);
  const int64_t whole = (n - head) * (int64_t)sizeof(O) / 16, tail = head + whole * 16 / (int64_t)sizeof(O);
  u32x4_t* const span = reinterpret_cast<u32x4_t*>(table + head);
  const u32x4_t zero = {0, 0, 0, 0};
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < whole; i += (int64_t)gridDim.x * kThreads)
    st_global<u32x4_t>(span + i, zero);
  if (blockIdx.x == 0) {
    if ((int64_t)threadIdx.x < head) table[threadIdx.x] = 0;
    if (tail + (int64_t)threadIdx.x < n) table[tail + threadIdx.x] = 0;
  }
}
template <typename O>
__global__ __launch_bounds__(kThreads) void clear_rows_kernel(EmbeddingGradArgs p) {
  const float zeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x)
    for (int c = 8 * (int)threadIdx.x; c < (int)p.cols; c += 8 * kThreads)
      store8<O>(reinterpret_cast<O*>(p.dtable) + row * p.ldt, c, (int)p.cols, zeros);
}

// Up to 8192 or 16384 tokens: a token's place is the number of smaller keys, and of equal ones
// before it.  A workgroup ranks 32 tokens against all keys, 32 slices of them side by side.
// n^2 comparisons of about three instructions, but on all CUs, in one launch and without
// a pass per digit: 8192 tokens 10.3 us, bound by issue (a sort of 18 bits by one workgroup:
// 20.4).
template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_ranks_kernel(EmbeddingGradArgs p) {
  constexpr int kTokens = 32, kSlices = kSortThreads / kTokens;
  __shared__ __attribute__((aligned(16))) uint32_t keys[kSortThreads * kSortAlone];
  __shared__ uint32_t ranks[kTokens];
  const int n = (int)p.count, t = threadIdx.x % kTokens, slice = threadIdx.x / kTokens;
  const int size = (n + 4 * kSlices - 1) / (4 * kSlices) * 4, all = size * kSlices;
  constexpr int kAhead = 8;
  const I* tokens = reinterpret_cast<const I*>(p.tokens);
  for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kSortThreads) {
    I token[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) token[a] = ld_global<I>(tokens + min(i0 + a * kSortThreads, n - 1));
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kSortThreads;
      if (i < all) keys[i] = i < n ? key_of(p, token[a]) : 0xffffffffu;
    }
  }
  if (threadIdx.x < kTokens) ranks[threadIdx.x] = 0;
  __syncthreads();
  const int i = blockIdx.x * kTokens + t, first = slice * size;
  const uint32_t key = keys[min(i, n - 1)];
  const int before = min(max(i - first, 0), size);   // keys of the slice that stand before the token
  uint32_t rank = 0;
#pragma unroll 8
  for (int j = 0; j < size; j += 4) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(keys + first + j);
    const uint32_t behind = key + (j + 4 <= before ? 1 : 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) rank += v[e] < behind ? 1 : 0;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e) {   // the four that the token stands among
    const int j = (before & ~3) + e;
    if (j < before) rank += keys[first + j] == key ? 1 : 0;
  }
  atomicAdd(&ranks[t], rank);   // whole numbers: their order does not matter
  __syncthreads();
  if (slice == 0 && i < n) {
    p.keys[0][ranks[t]] = key;
    p.places[0][ranks[t]] = (uint32_t)i;
  }
}

// More tokens: per pass the digits' counts of every workgroup, where each begins, and
// the keys put there.  `from` is the buffer read (pass 0: the tokens).  20000 tokens, a pass:
// 6.0 + 10.0 us, latencies of 5 workgroups (18 us with a launch between for the beginnings,
// which more than 32 workgroups have).
__device__ __forceinline__ void read_keys(const EmbeddingGradArgs& p, int pass, int from, int64_t first,
                                          uint32_t (&key)[kSortBeside], uint32_t (&place)[kSortBeside]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < kSortBeside; ++k) {
    const int64_t i = first + wave * 64 * kSortBeside + k * 64 + lane;
    key[k] = place[k] = 0;
    if (i < p.count) {
      key[k] = pass == 0 ? key_of(p, token_at(p.tokens, p.wide, i)) : p.keys[from][i];
      place[k] = pass == 0 ? (uint32_t)i : p.places[from][i];
    }
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(EmbeddingGradArgs p, SortPlan plan, int pass, int from) {
  __shared__ uint32_t count[kSortDigits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)blockIdx.x * kSortBlock;
  uint32_t key[kSortBeside], place[kSortBeside];
  read_keys(p, pass, from, first, key, place);
  count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortBeside; ++k)   // whole numbers: their order does not matter
    if (first + wave * 64 * kSortBeside + k * 64 + lane < p.count)
      atomicAdd(&count[(key[k] >> (pass * plan.bits)) & ((1u << plan.bits) - 1)], 1u);
  __syncthreads();
  p.digits[(int64_t)blockIdx.x * kSortDigits + threadIdx.x] = count[threadIdx.x];
}
static_assert(kSortDigits == kSortThreads, "a thread per digit");

// The sum of the threads' values before this one's.
__device__ __forceinline__ uint32_t sum_before(uint32_t value, uint32_t (&sums)[kWaves]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t sum = value;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t up = __shfl_up(sum, off, 64);
    if (lane >= off) sum += up;
  }
  if (lane == 63) sums[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += sums[w];
  return sum - value;
}

// digits[block][d] -> where block's keys of digit d begin.
__global__ __launch_bounds__(kSortThreads) void sort_begin_kernel(EmbeddingGradArgs p, SortPlan plan) {
  __shared__ uint32_t sums[kWaves];
  const int d = threadIdx.x;
  const bool live = d < 1 << plan.bits;
  constexpr int kAhead = 16;
  uint32_t c[kAhead];
  auto load = [&](int64_t b0) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) c[b] = p.digits[min(b0 + b, plan.blocks - 1) * kSortDigits + d];
  };
  uint32_t total = 0;
  if (live)
    for (int64_t b0 = 0; b0 < plan.blocks; b0 += kAhead) {
      load(b0);
#pragma unroll
      for (int b = 0; b < kAhead; ++b) total += b0 + b < plan.blocks ? c[b] : 0;
    }
  uint32_t at = sum_before(total, sums);
  if (!live) return;
  for (int64_t b0 = 0; b0 < plan.blocks; b0 += kAhead) {
    load(b0);
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      if (b0 + b < plan.blocks) p.digits[(b0 + b) * kSortDigits + d] = at;
      at += c[b];
    }
  }
}

// OWN: each workgroup finds by itself where its keys begin, from the counts.
template <bool OWN>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(EmbeddingGradArgs p, SortPlan plan, int pass, int from, int to) {
  __shared__ SortLds lds;
  __shared__ uint32_t sums[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)blockIdx.x * kSortBlock;
  uint32_t key[kSortBeside], place[kSortBeside], rank[kSortBeside];
  read_keys(p, pass, from, first, key, place);
  const int shift = pass * plan.bits;
  const uint32_t mask = (1u << plan.bits) - 1;
  count_digits<kSortBeside>(lds, key, rank, p.count - first, shift, plan.bits);
  // before this wavefront's keys of a digit: the other workgroups' and wavefronts'
  const int d = threadIdx.x;
  uint32_t at = 0;
  if constexpr (OWN) {
    uint32_t all = 0;
    constexpr int kAhead = 8;
    for (int b0 = 0; b0 < (int)plan.blocks; b0 += kAhead) {
      uint32_t c[kAhead];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) c[b] = p.digits[min(b0 + b, (int)plan.blocks - 1) * kSortDigits + d];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        all += b0 + b < (int)plan.blocks ? c[b] : 0;
        at += b0 + b < (int)blockIdx.x ? c[b] : 0;
      }
    }
    at += sum_before(all, sums);
  } else if (d <= (int)mask) {
    at = p.digits[(int64_t)blockIdx.x * kSortDigits + d];
  }
  if (d <= (int)mask) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = lds.count[w][d];
      lds.count[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortBeside; ++k)
    if (first + wave * 64 * kSortBeside + k * 64 + lane < p.count) {
      const uint32_t at = lds.count[wave][(key[k] >> shift) & mask] + rank[k];
      p.keys[to][at] = key[k];
      p.places[to][at] = place[k];
    }
}

// A row of the table's gradient: 8 columns of it, rounded once.
template <typename O>
__device__ __forceinline__ void store_sum(const EmbeddingGradArgs& p, uint32_t key, int c, const float (&sum)[8]) {
  if (key >= (uint32_t)p.rows) return;
  O* dst = reinterpret_cast<O*>(p.dtable) + (int64_t)key * p.ldt;
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = sum[j] * p.scale;
  if (p.accumulate) {
    float old[8];
    load8<O>(dst, c, (int)p.cols).widen(old);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += old[j];
  }
  store8<O>(dst, c, (int)p.cols, a);
}
// load8 of one chunk of many rows: first all loads, then what belongs to a row's end.
struct Chunk {
  int c, cols, skip;   // skip: elements before c that the load of a row's last eight has
  __device__ __forceinline__ Chunk(int c, int cols) : c(c), cols(cols), skip(cols >= 8 ? max(c + 8 - cols, 0) : 0) {}
  template <typename T>
  __device__ __forceinline__ void load(Raw8<T>& r, const T* row) const {
    if (cols >= 8) r.load(row + c - skip);
    else r = load8<T>(row, c, cols);
  }
  template <typename T>
  __device__ __forceinline__ void widen(Raw8<T>& r, float (&v)[8]) const {
    if (skip > 0) r.drop(skip);
    r.widen(v);
  }
};
__device__ __forceinline__ void store_partial(float* row, int c, int cols, const float (&sum)[8]) {
  store8<float>(row, c, cols, sum);
}

// Sums of a run of sorted tokens: rows whose tokens all lie in the run are written,
// the sums of the row that began before it and of the one that goes on behind it are
// left in partials[run][0] and [1] (one that does both: in [0]).  Runs are short, so that
// there are enough workgroups, and their rows are all on their way at once: 8192 x 2048 bf16
// 24 us, 20000 x 769 bf16 11.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void embedding_sum_kernel(EmbeddingGradArgs p, int which, int log_group, int64_t run) {
  const int group = 1 << log_group, t = threadIdx.x & (group - 1);
  const int64_t r = (int64_t)blockIdx.x * (kThreads >> log_group) + (threadIdx.x >> log_group);
  const int64_t first = r * run, end = min(first + run, p.count);
  const int c = 8 * ((int)blockIdx.y * group + t), cols = (int)p.cols;
  if (first >= p.count || c >= cols) return;
  const uint32_t* keys = p.keys[which];
  const uint32_t* places = p.places[which];
  float* part = p.partials + r * 2 * p.cols;
  const T* dout = reinterpret_cast<const T*>(p.dout);
  const uint32_t before = first > 0 ? keys[first - 1] : 0xffffffffu, behind = end < p.count ? keys[end] : 0xffffffffu;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  const Chunk chunk(c, cols);
  uint32_t current = keys[first];
  bool opened = current == before;   // the current row's tokens began in an earlier run
  constexpr int kAhead = sizeof(T) == 2 ? 16 : 8;   // bf16: all rows of a short run are on their way at once
  for (int64_t i = first; i < end; i += kAhead) {
    Raw8<T> v[kAhead];
    uint32_t key[kAhead], place[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t at = min(i + a, end - 1);
      key[a] = keys[at];
      place[a] = places[at];
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) chunk.load(v[a], dout + (int64_t)place[a] * p.ldd);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i + a >= end) break;
      if (key[a] != current) {
        if (opened) store_partial(part, c, cols, sum);
        else store_sum<O>(p, current, c, sum);
        opened = false;
        current = key[a];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
      }
      float x[8];
      chunk.widen(v[a], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += x[j];
    }
  }
  if (opened) store_partial(part, c, cols, sum);
  else if (current == behind) store_partial(part + p.cols, c, cols, sum);
  else store_sum<O>(p, current, c, sum);
}

// Joins the partial sums of a row whose tokens begin in run r and go on: its runs are
// counted by the workgroup's threads side by side, then 8 groups of 32 threads add every
// eighth run's sums, four at a time, and those are added in order (eight at a time are 0.5 to
// 1.5 us slower).  20000 tokens of 300 rows: 9 us, the latency of about five loads that wait for
// each other in the most frequent row's.
constexpr int kJoin = 8;
template <typename O>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(EmbeddingGradArgs p, int which, int64_t run) {
  __shared__ float sums[kJoin][32][9];
  const int64_t r = blockIdx.x, first = r * run, end = first + run;
  if (end >= p.count) return;
  const uint32_t* keys = p.keys[which];
  const uint32_t key = keys[end - 1], behind = keys[end], before = first > 0 ? keys[first - 1] : 0xffffffffu;
  // a row of several runs that began before this one is joined by the run it began in
  if (behind != key || key >= (uint32_t)p.rows || before == key) return;
  const int64_t runs = (p.count + run - 1) / run;
  int64_t last = r + 1;   // the last run that begins with the key
  for (;;) {
    const int64_t q = last + 1 + threadIdx.x;
    const int more = __syncthreads_count(q < runs && keys[min(q, runs - 1) * run] == key);
    last += more;
    if (more < kThreads) break;
  }
  const int t = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = 8 * ((int)blockIdx.y * 32 + t), cols = (int)p.cols;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  constexpr int kAhead = 4;
  const Chunk chunk(c, cols);
  if (c < cols)
    for (int64_t q = r + g; q <= last; q += kAhead * kJoin) {
      Raw8<float> v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int64_t at = q + a * kJoin;
        v[a].zero();
        if (at <= last) chunk.load(v[a], p.partials + (at * 2 + (at == r)) * p.cols);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        float x[8];
        chunk.widen(v[a], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += x[j];
      }
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[g][t][j] = sum[j];
  __syncthreads();
  if (g != 0 || c >= cols) return;
#pragma unroll
  for (int q = 1; q < kJoin; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += sums[q][t][j];
  store_sum<O>(p, key, c, sum);
}

// Threads per row, as a power of two's exponent: as many as it has vectors, at most 256.
int log_group_of(int64_t cols) {
  int g = 0;
  while (g < 8 && ((int64_t)8 << g) < cols) ++g;
  return g;
}

template <typename T, typename O>
hipError_t backward_for(const EmbeddingGradArgs& a, hipStream_t st) {
  const SortPlan plan = plan_sort(a.count, a.rows);
  hipError_t e = hipSuccess;
  if (!a.accumulate) {
    if (a.ldt == a.cols || a.rows == 1) {
      const int64_t groups = (a.rows * a.cols * (int64_t)sizeof(O) / 16 + kThreads - 1) / kThreads;
      hipLaunchKernelGGL(clear_kernel<O>, dim3((unsigned)std::min(std::max<int64_t>(groups, 1), kClearGroups)), dim3(kThreads), 0, st, a);
    } else {
      hipLaunchKernelGGL(clear_rows_kernel<O>, dim3((unsigned)std::min(a.rows, kClearGroups)), dim3(kThreads), 0, st, a);
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.count == 0) return e;
  int which = 0;
  if (plan.blocks == 1) {
    const dim3 grid((unsigned)((a.count + 31) / 32)), block(kSortThreads);
    if (a.wide) hipLaunchKernelGGL(sort_ranks_kernel<int64_t>, grid, block, 0, st, a);
    else hipLaunchKernelGGL(sort_ranks_kernel<int32_t>, grid, block, 0, st, a);
  } else {
    const dim3 grid((unsigned)plan.blocks), block(kSortThreads);
    for (int pass = 0; pass < plan.passes; ++pass) {
      const int from = which;
      which = pass == 0 ? 0 : 1 - which;
      hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, st, a, plan, pass, from);
      if (plan.blocks <= kOwnBegin) {
        hipLaunchKernelGGL(sort_place_kernel<true>, grid, block, 0, st, a, plan, pass, from, which);
      } else {
        hipLaunchKernelGGL(sort_begin_kernel, dim3(1), block, 0, st, a, plan);
        hipLaunchKernelGGL(sort_place_kernel<false>, grid, block, 0, st, a, plan, pass, from, which);
      }
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int lg = log_group_of(a.cols);
  const int64_t run = sum_run(a.count), runs = (a.count + run - 1) / run, per = kThreads >> lg;
  const unsigned wide = (unsigned)((a.cols + (8 << lg) - 1) / (8 << lg));
  hipLaunchKernelGGL((embedding_sum_kernel<T, O>), dim3((unsigned)((runs + per - 1) / per), wide), dim3(kThreads), 0, st,
                     a, which, lg, run);
  e = hipGetLastError();
  if (e != hipSuccess || runs < 2) return e;
  hipLaunchKernelGGL(embedding_join_kernel<O>, dim3((unsigned)(runs - 1), (unsigned)((a.cols + 255) / 256)), dim3(kThreads),
                     0, st, a, which, run);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding_forward(int table_bf16, int out_bf16, const EmbeddingArgs& a, hipStream_t st) {
  const int lg = log_group_of(a.cols);
  const int64_t per = kThreads >> lg;
  const dim3 grid((unsigned)((a.count + per - 1) / per)), block(kThreads);
  if (table_bf16) {
    if (out_bf16) hipLaunchKernelGGL((embedding_forward_kernel<uint16_t, uint16_t>), grid, block, 0, st, a, lg);
    else hipLaunchKernelGGL((embedding_forward_kernel<uint16_t, float>), grid, block, 0, st, a, lg);
  } else {
    if (out_bf16) hipLaunchKernelGGL((embedding_forward_kernel<float, uint16_t>), grid, block, 0, st, a, lg);
    else hipLaunchKernelGGL((embedding_forward_kernel<float, float>), grid, block, 0, st, a, lg);
  }
  return hipGetLastError();
}

hipError_t launch_embedding_backward(int dout_bf16, int table_bf16, const EmbeddingGradArgs& a, hipStream_t st) {
  if (dout_bf16) return table_bf16 ? backward_for<uint16_t, uint16_t>(a, st) : backward_for<uint16_t, float>(a, st);
  return table_bf16 ? backward_for<float, uint16_t>(a, st) : backward_for<float, float>(a, st);
}

}  // namespace muonh
