// Drives the host code of the attention, the residual norm and the embedding
// (attention.cpp, add_norm.cpp, embedding.cpp) with no device: workspaces, refusals,
// calls that have nothing to do, and what the launchers are given.  Launchers are
// stubs that keep their arguments and report no device.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "../../pretraining_optimizer_amd/csrc/attention.h"
#include "../../pretraining_optimizer_amd/csrc/embedding.h"
#include "../../pretraining_optimizer_amd/csrc/operators.h"
#include "../../pretraining_optimizer_amd/csrc/step_tail.h"

using namespace muonh;

static std::string g_error;
static int g_launches;
static AttentionArgs g_attention;
static AttentionGradArgs g_attention_grad;
static AddNormArgs g_norm;
static QuantArgs g_norm_forms;
static NormGradArgs g_norm_grad;
static EmbeddingArgs g_embedding;
static EmbeddingGradArgs g_embedding_grad;

template <typename T>
static hipError_t keep(T& kept, const T& a) {
  kept = a;
  ++g_launches;
  return hipErrorNoDevice;
}

namespace muonh {
int set_last_error(int code, const char* msg) {
  g_error = msg;
  return code;
}
hipError_t launch_block_quantize(int, int, const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_block_matmul(int, const MatmulPlan&, const BlockMatmulArgs&, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_norm_forward(int, int, const NormArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm_backward(int, int, const NormGradArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t norm_partial_rows(int64_t rows, int64_t) { return rows < 256 ? rows : 256; }
bool add_norm_rows_quantize(int64_t cols) { return cols <= 16384; }
// the first of two launches: let the second one run
hipError_t launch_add_norm_rows(int, const AddNormArgs& a, hipStream_t) {
  (void)keep(g_norm, a);
  return hipSuccess;
}
hipError_t launch_norm_quantize(int, const QuantArgs& out, const float*, const float*, hipStream_t) {
  return keep(g_norm_forms, out);
}
hipError_t launch_add_norm_backward(int, const NormGradArgs& a, hipStream_t) { return keep(g_norm_grad, a); }
hipError_t launch_attention_forward(const AttentionArgs& a, hipStream_t) { return keep(g_attention, a); }
hipError_t launch_attention_backward(const AttentionGradArgs& a, hipStream_t) { return keep(g_attention_grad, a); }
hipError_t launch_embedding_forward(int, int, const EmbeddingArgs& a, hipStream_t) { return keep(g_embedding, a); }
hipError_t launch_embedding_backward(int, int, const EmbeddingGradArgs& a, hipStream_t) {
  return keep(g_embedding_grad, a);
}
}  // namespace muonh

#define CHECK(x)                                                             \
  do {                                                                       \
    if (!(x)) {                                                              \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, g_error.c_str());      \
      std::exit(1);                                                          \
    }                                                                        \
  } while (0)

// Addresses that no memory stands at, 2^38 bytes apart.
static char* at(int i) { return reinterpret_cast<char*>((uintptr_t)(i + 1) << 38); }
static float* vector_at(int i) { return reinterpret_cast<float*>(at(i)); }

static muonh_attention_args attention_args(int64_t tokens, int64_t sequences, int32_t heads, int32_t kv_heads, int32_t dim) {
  muonh_attention_args a{};
  a.q = at(0);
  a.k = at(1);
  a.v = at(2);
  a.out = at(3);
  a.lse = vector_at(4);
  a.cu_seqlens = reinterpret_cast<const int32_t*>(at(5));
  a.ld_q = a.ld_out = (int64_t)heads * dim;
  a.ld_k = a.ld_v = (int64_t)kv_heads * dim;
  a.tokens = tokens;
  a.sequences = sequences;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.scale = 0.1f;
  return a;
}

static void attention() {
  const int64_t counts[] = {0, 1, 31, 32, 127, 128, 129, 8192, 1 << 20, 1 << 30};
  const int64_t sequences[] = {0, 1, 2, 63, 64, 65, 4096, 1 << 20, 1 << 30};
  int ran = 0, refused = 0;
  for (int64_t t : counts)
    for (int64_t s : sequences)
      for (int32_t heads : {1, 3, 24, 128, 65535})
        for (int32_t dim : {8, 64, 128}) {
          muonh_attention_args a = attention_args(t, s, heads, 1, dim);
          size_t need = 12345;
          const int rc = muonh_attention_backward_workspace(&a, &need);
          const bool wide = a.ld_q > (1 << 23) - 1;
          if (rc != MUONH_OK) {
            CHECK(rc == MUONH_EINVAL && need == 12345);
            CHECK(muonh_attention_forward(&a, nullptr) == MUONH_EINVAL);
            ++refused;
            continue;
          }
          CHECK(need == (s == 0 ? 0 : 2 * (((size_t)heads * (size_t)t * 4 + 255) / 256 * 256)));
          const int before = g_launches;
          const bool far = (double)t * (double)a.ld_q * 2.0 > (double)((int64_t)1 << 38);   // into the next address
          const int f = muonh_attention_forward(&a, nullptr);
          if (wide)
            CHECK(f == MUONH_EINVAL && g_launches == before);
          else if (t == 0 || s == 0)
            CHECK(f == MUONH_OK && g_launches == before);
          else if (!far)
            CHECK(f == MUONH_EHIP && g_launches == before + 1 && g_attention.tokens == t);
          ++ran;
        }
  CHECK(ran > 0 && refused > 0);

  muonh_attention_args good = attention_args(1000, 2, 8, 2, 64);
  auto refuses = [&](auto change, const char* text) {
    muonh_attention_args a = good;
    change(a);
    const int before = g_launches;
    const int rc = muonh_attention_forward(&a, nullptr);
    return rc == MUONH_EINVAL && g_launches == before && g_error.find(text) != std::string::npos;
  };
  using A = muonh_attention_args;
  CHECK(refuses([](A& a) { a.heads = 7; }, "multiple of kv_heads"));
  CHECK(refuses([](A& a) { a.kv_heads = 0; }, "multiple of kv_heads"));
  CHECK(refuses([](A& a) { a.kv_heads = -2; }, "multiple of kv_heads"));
  CHECK(refuses([](A& a) { a.dim = 12; }, "dim"));
  CHECK(refuses([](A& a) { a.dim = 136; }, "dim"));
  CHECK(refuses([](A& a) { a.scale = 0.0f; }, "scale"));
  CHECK(refuses([](A& a) { a.scale = NAN; }, "scale"));
  CHECK(refuses([](A& a) { a.scale = INFINITY; }, "scale"));
  CHECK(refuses([](A& a) { a.tokens = -1; }, "tokens"));
  CHECK(refuses([](A& a) { a.sequences = ((int64_t)1 << 30) + 1; }, "sequences"));
  CHECK(refuses([](A& a) { a.ld_q = 508; }, "q: the pitch"));
  CHECK(refuses([](A& a) { a.ld_k = 120; }, "k: the pitch"));
  CHECK(refuses([](A& a) { a.ld_v = 1 << 23; }, "v: the pitch"));
  CHECK(refuses([](A& a) { a.ld_out = 516; }, "out: the pitch"));
  CHECK(refuses([](A& a) { a.q = nullptr; }, "null pointer: q"));
  CHECK(refuses([](A& a) { a.k = at(1) + 8; }, "k must be 16-byte aligned"));
  CHECK(refuses([](A& a) { a.lse = nullptr; }, "lse or cu_seqlens"));
  CHECK(refuses([](A& a) { a.cu_seqlens = reinterpret_cast<const int32_t*>(at(5) + 2); }, "misaligned"));
  CHECK(refuses([](A& a) { a.out = at(0); }, "out overlaps q"));
  CHECK(refuses([](A& a) { a.out = at(2) + 16; }, "out overlaps v"));
  CHECK(refuses([](A& a) { a.lse = vector_at(3) + 4; }, "lse"));
  CHECK(refuses([](A& a) { a.lse = vector_at(1) + 4; }, "lse"));
  // inputs and the output side by side in rows of one pitch; one column too near
  muonh_attention_args side = good;
  side.ld_q = side.ld_k = side.ld_v = side.ld_out = 512 + 128 + 128 + 512;
  side.k = at(0) + 512 * 2;
  side.v = at(0) + (512 + 128) * 2;
  side.out = at(0) + (512 + 256) * 2;
  CHECK(muonh_attention_forward(&side, nullptr) == MUONH_EHIP);
  side.out = at(0) + (512 + 256 - 8) * 2;
  CHECK(muonh_attention_forward(&side, nullptr) == MUONH_EINVAL);

  muonh_attention_grad_args b{};
  b.a = good;
  b.dout = at(6);
  b.dq = at(7);
  b.dk = at(8);
  b.dv = at(9);
  b.ld_dout = b.ld_dq = 512;
  b.ld_dk = b.ld_dv = 128;
  size_t need = 0;
  CHECK(muonh_attention_backward_workspace(&good, &need) == MUONH_OK && need == 2 * 32000);
  b.workspace = at(10);
  b.workspace_bytes = need;
  CHECK(muonh_attention_backward(&b, nullptr) == MUONH_EHIP);
  CHECK((char*)g_attention_grad.row_lse == at(10) && (char*)g_attention_grad.row_delta == at(10) + 32000);
  auto refuses_back = [&](auto change, int code, const char* text) {
    muonh_attention_grad_args a = b;
    change(a);
    const int before = g_launches;
    const int rc = muonh_attention_backward(&a, nullptr);
    return rc == code && g_launches == before && g_error.find(text) != std::string::npos;
  };
  using B = muonh_attention_grad_args;
  CHECK(refuses_back([](B& a) { a.workspace_bytes -= 1; }, MUONH_ENOMEM, "workspace too small"));
  CHECK(refuses_back([](B& a) { a.workspace = nullptr; }, MUONH_ENOMEM, "workspace too small"));
  CHECK(refuses_back([](B& a) { a.workspace = at(10) + 16; }, MUONH_EINVAL, "256-byte"));
  CHECK(refuses_back([](B& a) { a.workspace = at(7); }, MUONH_EINVAL, "overlaps"));
  CHECK(refuses_back([](B& a) { a.workspace = at(6); }, MUONH_EINVAL, "overlaps"));
  CHECK(refuses_back([](B& a) { a.workspace = at(4); }, MUONH_EINVAL, "overlap"));
  CHECK(refuses_back([](B& a) { a.dk = at(1); }, MUONH_EINVAL, "dk overlaps k"));
  CHECK(refuses_back([](B& a) { a.dq = at(6); }, MUONH_EINVAL, "dq overlaps dout"));
  CHECK(refuses_back([](B& a) { a.dv = at(8) + 128; }, MUONH_EINVAL, "dk overlaps dv"));
  CHECK(refuses_back([](B& a) { a.dout = nullptr; }, MUONH_EINVAL, "null pointer: dout"));
  CHECK(refuses_back([](B& a) { a.ld_dv = 132; }, MUONH_EINVAL, "dv: the pitch"));
  CHECK(muonh_attention_forward(nullptr, nullptr) == MUONH_EINVAL && muonh_attention_backward(nullptr, nullptr) == MUONH_EINVAL);
  b.a.sequences = 0;
  b.workspace = nullptr;
  CHECK(muonh_attention_backward(&b, nullptr) == MUONH_OK);
}

static muonh_fp8_matrix form(int64_t rows, int64_t cols, char* data) {
  return muonh_fp8_matrix{data, data + ((uintptr_t)1 << 36), rows, cols, (cols + 127) / 128 * 128,
                          (cols + 511) / 512 * 4, 1, 0};
}

static void residual_norm() {
  muonh_add_norm_args g{};
  g.x = at(0);
  g.residual = at(1);
  g.weight = vector_at(2);
  g.h = at(3);
  g.rstd = vector_at(4);
  g.rows = 300;
  g.cols = 500;
  g.ldx = g.ld_residual = g.ldh = 504;
  g.dtype = MUONH_BF16;
  g.eps = 1e-6f;
  muonh_fp8_matrix q = form(300, 500, at(5)), qt = form(500, 300, at(6));
  int before = g_launches;
  CHECK(muonh_add_norm_quantize(&g, &q, &qt, nullptr) == MUONH_EHIP && g_launches == before + 2);
  // the first launch writes the row form, the second one the column form
  CHECK(g_norm.q == (uint8_t*)at(5) && !g_norm_forms.q && g_norm_forms.qt == (uint8_t*)at(6) && g_norm_forms.x == at(3));
  before = g_launches;
  CHECK(muonh_add_norm_quantize(&g, &q, nullptr, nullptr) == MUONH_OK && g_launches == before + 1);
  muonh_add_norm_args wide = g;
  wide.cols = wide.ldx = wide.ld_residual = wide.ldh = 20000;
  muonh_fp8_matrix wq = form(300, 20000, at(5));
  CHECK(muonh_add_norm_quantize(&wide, &wq, nullptr, nullptr) == MUONH_EHIP);
  CHECK(!g_norm.q && g_norm_forms.q == (uint8_t*)at(5) && !g_norm_forms.qt);
  muonh_add_norm_args alone = g;
  alone.residual = alone.h = nullptr;
  CHECK(muonh_add_norm_quantize(&alone, nullptr, &qt, nullptr) == MUONH_EHIP && g_norm_forms.x == at(0));
  auto refuses = [&](auto change, const char* text) {
    muonh_add_norm_args a = g;
    muonh_fp8_matrix aq = q, aqt = qt;
    change(a, aq, aqt);
    const int n = g_launches;
    const int rc = muonh_add_norm_quantize(&a, &aq, &aqt, nullptr);
    return rc == MUONH_EINVAL && g_launches == n && g_error.find(text) != std::string::npos;
  };
  using A = muonh_add_norm_args;
  using Q = muonh_fp8_matrix;
  CHECK(refuses([](A& a, Q&, Q&) { a.residual = nullptr; }, "h must be NULL"));
  CHECK(refuses([](A& a, Q&, Q&) { a.h = nullptr; }, "null pointer"));
  CHECK(refuses([](A& a, Q&, Q&) { a.eps = -1.0f; }, "eps"));
  CHECK(refuses([](A& a, Q&, Q&) { a.eps = NAN; }, "eps"));
  CHECK(refuses([](A& a, Q&, Q&) { a.cols = 0; }, "cols"));
  CHECK(refuses([](A& a, Q&, Q&) { a.ldh = 499; }, "ldh"));
  CHECK(refuses([](A&, Q& x, Q&) { x.rows = 299; }, "q: shape"));
  CHECK(refuses([](A&, Q&, Q& y) { y.block_rows = 128; }, "qt: block_rows"));
  CHECK(refuses([](A&, Q&, Q& y) { y.data = at(5) + 512; }, "overlaps"));
  CHECK(refuses([](A&, Q& x, Q&) { x.scale = at(5) + 512; }, "overlaps"));
  CHECK(refuses([](A&, Q& x, Q&) { x.data = at(0); }, "overlaps"));
  CHECK(refuses([](A&, Q& x, Q&) { x.data = at(3) + 512; }, "overlaps"));
  CHECK(refuses([](A& a, Q&, Q&) { a.h = at(0) + 2; }, "h overlaps"));
  CHECK(refuses([](A& a, Q&, Q&) { a.rstd = vector_at(2) + 8; }, "overlaps"));
  CHECK(refuses([](A& a, Q&, Q&) { a.x = at(0) + 1; }, "misaligned"));
  before = g_launches;
  CHECK(muonh_add_norm_quantize(&g, nullptr, nullptr, nullptr) == MUONH_EINVAL && g_launches == before);
  muonh_add_norm_args in_place = g;
  in_place.h = at(1);
  CHECK(muonh_add_norm_quantize(&in_place, &q, &qt, nullptr) == MUONH_EHIP);
  muonh_add_norm_args none = g;
  none.rows = 0;
  muonh_fp8_matrix q0 = form(0, 500, at(5)), qt0 = form(500, 0, at(6));
  qt0.ld = 128;
  qt0.ld_scale = 4;
  before = g_launches;
  CHECK(muonh_add_norm_quantize(&none, &q0, &qt0, nullptr) == MUONH_OK && g_launches == before);

  muonh_add_norm_grad_args b{};
  b.g.dy = at(0);
  b.g.x = at(1);
  b.g.weight = vector_at(2);
  b.g.rstd = vector_at(3);
  b.g.dx = at(4);
  b.g.dweight = vector_at(5);
  b.g.rows = 300;
  b.g.cols = 500;
  b.g.ld_dy = b.g.ldx = b.g.ld_dx = b.ld_dh = 500;
  b.g.dtype = MUONH_BF16;
  b.g.kind = MUONH_NORM_RMS;
  b.dh = at(6);
  size_t need = 0;
  CHECK(muonh_norm_backward_workspace(300, 500, &need) == MUONH_OK && need > 0);
  b.g.workspace = at(7);
  b.g.workspace_bytes = need;
  CHECK(muonh_add_norm_backward(&b, nullptr) == MUONH_EHIP && g_norm_grad.dh == at(6) && g_norm_grad.lddh == 500);
  auto refuses_back = [&](auto change, int code, const char* text) {
    muonh_add_norm_grad_args a = b;
    change(a);
    const int n = g_launches;
    const int rc = muonh_add_norm_backward(&a, nullptr);
    return rc == code && g_launches == n && g_error.find(text) != std::string::npos;
  };
  using B = muonh_add_norm_grad_args;
  CHECK(refuses_back([](B& a) { a.g.kind = MUONH_NORM_LAYER; }, MUONH_EINVAL, "kind"));
  CHECK(refuses_back([](B& a) { a.dh = nullptr; }, MUONH_EINVAL, "null pointer"));
  CHECK(refuses_back([](B& a) { a.g.mean = vector_at(9); }, MUONH_EINVAL, "mean and dbias"));
  CHECK(refuses_back([](B& a) { a.ld_dh = 499; }, MUONH_EINVAL, "ld_dh"));
  CHECK(refuses_back([](B& a) { a.g.workspace_bytes -= 1; }, MUONH_ENOMEM, "workspace"));
  CHECK(refuses_back([](B& a) { a.g.workspace = at(6) + 256; }, MUONH_EINVAL, "overlaps"));
  CHECK(refuses_back([](B& a) { a.g.dx = at(6) + 2; }, MUONH_EINVAL, "dx overlaps"));
  CHECK(refuses_back([](B& a) { a.g.dweight = vector_at(6); }, MUONH_EINVAL, "overlaps"));
  CHECK(refuses_back([](B& a) { a.g.accumulate = 2; }, MUONH_EINVAL, "accumulate"));
  b.g.dx = at(6);   // in place of dh
  CHECK(muonh_add_norm_backward(&b, nullptr) == MUONH_EHIP);
}

static void embedding() {
  // sort plans and workspaces: every token in a block, every bit of a key in a pass
  const int64_t counts[] = {0, 1, 16, 17, 8192, 8193, 65536, 65537, 1000000, (int64_t)1 << 30};
  const int64_t rows[] = {0, 1, 2, 300, 1023, 1024, 151936, 1 << 20, 1 << 30};
  int ran = 0, refused = 0;
  for (int64_t n : counts)
    for (int64_t r : rows)
      for (int64_t cols : {(int64_t)1, (int64_t)769, (int64_t)2048, (int64_t)1 << 20}) {
        size_t need = 777;
        const int rc = muonh_embedding_backward_workspace(n, r, cols, &need);
        if (rc != MUONH_OK) {
          CHECK(rc == MUONH_EINVAL && need == 777 && n * ((cols + 255) / 256 * 256) > 0xffffffffLL);
          ++refused;
          continue;
        }
        ++ran;
        CHECK(need % 256 == 0 && (n > 0) == (need > 0));
        if (n == 0) continue;
        const SortPlan p = plan_sort(n, r);
        CHECK(p.bits >= 1 && p.bits <= 10 && ((int64_t)1 << p.bits) <= kSortDigits);
        CHECK(((int64_t)1 << (p.bits * p.passes)) > r);
        CHECK(p.blocks == 1 ? n <= kSortThreads * kSortAlone && (p.passes > 1 || n <= 8192) : n > 8192 && p.blocks * kSortBlock >= n && (p.blocks - 1) * kSortBlock < n);
        const int64_t runs = (n + sum_run(n) - 1) / sum_run(n);
        CHECK((int64_t)need >= 16 * n + (runs > 1 ? runs * 2 * cols * 4 : 0));
        if (r == 0 || r * cols * 4 > ((int64_t)1 << 38) || n * cols * 2 > ((int64_t)1 << 38)) continue;
        muonh_embedding_grad_args b{};
        b.tokens = at(0);
        b.dout = at(1);
        b.dtable = at(2);
        b.count = n;
        b.rows = r;
        b.cols = b.ld_table = b.ld_dout = cols;
        b.token_bytes = 8;
        b.scale = 1.0f;
        b.dout_dtype = MUONH_BF16;
        b.table_dtype = MUONH_F32;
        b.workspace = at(8);
        b.workspace_bytes = need;
        CHECK(muonh_embedding_backward(&b, nullptr) == MUONH_EHIP);
        // the parts in order, each from behind the one before it
        const EmbeddingGradArgs& a = g_embedding_grad;
        const char* parts[] = {(char*)a.keys[0], (char*)a.places[0], (char*)a.keys[1], (char*)a.places[1], (char*)a.digits};
        CHECK(parts[0] == at(8));
        for (int i = 0; i < 4; ++i) CHECK(parts[i + 1] - parts[i] >= n * 4 && (uintptr_t)parts[i + 1] % 256 == 0);
        CHECK((char*)a.partials - (char*)a.digits >= (p.blocks > 1 ? p.blocks * kSortDigits * 4 : 0));
        CHECK((runs > 1 ? runs * 2 * cols * 4 : 0) <= at(8) + need - (char*)a.partials);
        b.workspace_bytes -= 1;
        CHECK(muonh_embedding_backward(&b, nullptr) == MUONH_ENOMEM);
      }
  CHECK(ran > 0 && refused > 0);

  muonh_embedding_args g{};
  g.tokens = at(0);
  g.table = at(1);
  g.out = at(2);
  g.count = 77;
  g.rows = 1000;
  g.cols = g.ld_table = g.ld_out = 777;
  g.token_bytes = 4;
  g.table_dtype = MUONH_F32;
  g.out_dtype = MUONH_BF16;
  g.scale = 2.0f;
  CHECK(muonh_embedding_forward(&g, nullptr) == MUONH_EHIP && g_embedding.count == 77 && !g_embedding.wide);
  auto refuses = [&](auto change, const char* text) {
    muonh_embedding_args a = g;
    change(a);
    const int n = g_launches;
    const int rc = muonh_embedding_forward(&a, nullptr);
    return rc == MUONH_EINVAL && g_launches == n && g_error.find(text) != std::string::npos;
  };
  using A = muonh_embedding_args;
  CHECK(refuses([](A& a) { a.token_bytes = 2; }, "token_bytes"));
  CHECK(refuses([](A& a) { a.scale = INFINITY; }, "scale"));
  CHECK(refuses([](A& a) { a.cols = 0; }, "cols"));
  CHECK(refuses([](A& a) { a.cols = ((int64_t)1 << 20) + 1; }, "cols"));
  CHECK(refuses([](A& a) { a.count = -1; }, "count"));
  CHECK(refuses([](A& a) { a.ld_out = 776; }, "ld_out"));
  CHECK(refuses([](A& a) { a.table = nullptr; }, "null pointer"));
  CHECK(refuses([](A& a) { a.tokens = at(0) + 2; }, "misaligned"));
  CHECK(refuses([](A& a) { a.out = at(1) + 4; }, "out overlaps"));
  CHECK(refuses([](A& a) { a.out_dtype = 7; }, "out: dtype"));
  const int before = g_launches;
  g.count = 0;
  CHECK(muonh_embedding_forward(&g, nullptr) == MUONH_OK && g_launches == before);
  muonh_embedding_grad_args b{};
  b.dtable = at(2);
  b.rows = 1000;
  b.cols = b.ld_table = b.ld_dout = 777;
  b.token_bytes = 8;
  b.scale = 1.0f;
  b.dout_dtype = b.table_dtype = MUONH_F32;
  b.accumulate = 1;
  CHECK(muonh_embedding_backward(&b, nullptr) == MUONH_OK && g_launches == before);   // nothing to add
  b.accumulate = 0;
  CHECK(muonh_embedding_backward(&b, nullptr) == MUONH_EHIP && g_launches == before + 1);   // cleared
  b.reserved = 1;
  CHECK(muonh_embedding_backward(&b, nullptr) == MUONH_EINVAL);
}

int main() {
  attention();
  residual_norm();
  embedding();
  std::printf("all checks passed\n");
  return 0;
}
