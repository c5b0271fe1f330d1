// Host side of the attention: argument checks, the workspace's size and the
// launches.  These entry points keep no state.

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "attention.h"
#include "operator_checks.h"
#include "operators.h"

using namespace muonh;

namespace {

constexpr int64_t kMaxPitch = ((int64_t)1 << 23) - 1;   // 128 rows stay below 2^31 bytes

constexpr int32_t kZeroResults = MUONH_ZERO_OUT | MUONH_ZERO_LSE, kZeroGradients = MUONH_ZERO_DQ | MUONH_ZERO_DK | MUONH_ZERO_DV;

// A tensor [tokens, cols] of bf16 with ld elements between tokens.
struct Tensor {
  const void* p;
  int64_t ld, cols;
  const char* name;
};

// Whether two tensors share no element: apart, or side by side in rows of one pitch.
bool separate(const Tensor& a, const Tensor& b, int64_t rows) {
  if (!overlap(a.p, extent(rows, a.cols, a.ld, 2), b.p, extent(rows, b.cols, b.ld, 2))) return true;
  if (a.ld != b.ld || rows == 1) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const Tensor &lo = x < y ? a : b, &hi = x < y ? b : a;
  const int64_t d = (int64_t)(x < y ? y - x : x - y) % (a.ld * 2);
  return d >= lo.cols * 2 && a.ld * 2 - d >= hi.cols * 2;
}

int check_tensor(const Tensor& t) {
  const std::string who = t.name;
  if (t.ld < t.cols || t.ld > kMaxPitch || t.ld % 8 != 0)
    return fail(MUONH_EINVAL, who + ": the pitch must be a multiple of 8, no less than a row and below 2^23");
  return MUONH_OK;
}
int check_address(const Tensor& t) {
  if (!t.p) return fail(MUONH_EINVAL, std::string("null pointer: ") + t.name);
  if (!aligned(t.p, 16)) return fail(MUONH_EINVAL, std::string(t.name) + " must be 16-byte aligned");
  return MUONH_OK;
}

int check_shape(const muonh_attention_args& g) {
  int rc;
  if ((rc = check_size(g.tokens, 0, "tokens")) || (rc = check_size(g.sequences, 0, "sequences"))) return rc;
  if (g.kv_heads < 1 || g.heads < 1 || g.heads % g.kv_heads != 0)
    return fail(MUONH_EINVAL, "heads must be a multiple of kv_heads, both at least 1");
  if (g.dim < 8 || g.dim > 128 || g.dim % 8 != 0) return fail(MUONH_EINVAL, "dim must be 8, 16, .. 128");
  if (!(g.scale > 0.0f) || !std::isfinite(g.scale)) return fail(MUONH_EINVAL, "scale must be > 0 and finite");
  if (g.zero_rest & ~(kZeroResults | kZeroGradients)) return fail(MUONH_EINVAL, "zero_rest must be a sum of MUONH_ZERO_*");
  if (g.reserved != 0) return fail(MUONH_EINVAL, "reserved != 0");
  if (attention_blocks(g.tokens, g.sequences + (g.zero_rest != 0), kAttentionRows) * 2 * kAttentionThreads > kMaxThreads / g.heads)
    return fail(MUONH_EINVAL, "tokens, sequences and heads are too many for one launch");
  return MUONH_OK;
}

size_t row_bytes(const muonh_attention_args& g) { return (size_t)(g.heads * g.tokens) * sizeof(float); }
// Whether a call writes nothing; `zeros` are its results' bits of zero_rest.
bool nothing_to_do(const muonh_attention_args& g, int32_t zeros) {
  return g.tokens == 0 || (g.sequences == 0 && !(g.zero_rest & zeros));
}
// Two rows of floats per head, each from a multiple of 256 bytes on.
size_t workspace_of(const muonh_attention_args& g) {
  return g.sequences == 0 ? 0 : 2 * (size_t)ceil_div((int64_t)row_bytes(g), kAlign) * kAlign;
}

AttentionArgs device_args(const muonh_attention_args& g, int32_t zeros) {
  AttentionArgs a{};
  a.q = static_cast<const uint16_t*>(g.q);
  a.k = static_cast<const uint16_t*>(g.k);
  a.v = static_cast<const uint16_t*>(g.v);
  a.out = static_cast<uint16_t*>(g.out);
  a.lse = g.lse;
  a.cu = g.cu_seqlens;
  a.ldq = g.ld_q;
  a.ldk = g.ld_k;
  a.ldv = g.ld_v;
  a.ldo = g.ld_out;
  a.tokens = (int32_t)g.tokens;
  a.sequences = (int32_t)g.sequences;
  a.heads = g.heads;
  a.kv_heads = g.kv_heads;
  a.dim = g.dim;
  a.scale = g.scale;
  a.zero_rest = g.zero_rest & zeros;
  return a;
}

// Inputs and outputs of one call: outputs share nothing with inputs or each other.
int check_sharing(const Tensor* outs, int no, const Tensor* ins, int ni, int64_t rows, std::initializer_list<Span> vec_outs,
                  std::initializer_list<Span> vec_ins) {
  for (int i = 0; i < no; ++i) {
    const std::string who = std::string(outs[i].name) + " overlaps ";
    for (int j = 0; j < ni; ++j)
      if (!separate(outs[i], ins[j], rows)) return fail(MUONH_EINVAL, who + ins[j].name);
    for (int j = i + 1; j < no; ++j)
      if (!separate(outs[i], outs[j], rows)) return fail(MUONH_EINVAL, who + outs[j].name);
    const Span s{outs[i].p, extent(rows, outs[i].cols, outs[i].ld, 2)};
    if (clash({s}, vec_outs) || clash({s}, vec_ins))
      return fail(MUONH_EINVAL, who + "lse, cu_seqlens or the workspace");
  }
  for (const Span& o : vec_outs)
    for (int j = 0; j < ni; ++j)
      if (overlap(o.p, o.bytes, ins[j].p, extent(rows, ins[j].cols, ins[j].ld, 2)))
        return fail(MUONH_EINVAL, std::string("lse or the workspace overlaps ") + ins[j].name);
  if (clash(vec_outs, vec_ins)) return fail(MUONH_EINVAL, "lse, cu_seqlens and the workspace overlap");
  return MUONH_OK;
}

}  // namespace

extern "C" {

int muonh_attention_forward(const muonh_attention_args* g, void* stream) {
  return guarded([&]() -> int {
    if (!g) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_shape(*g))) return rc;
    const int64_t cols = (int64_t)g->heads * g->dim, kv_cols = (int64_t)g->kv_heads * g->dim;
    const Tensor ins[] = {{g->q, g->ld_q, cols, "q"}, {g->k, g->ld_k, kv_cols, "k"}, {g->v, g->ld_v, kv_cols, "v"}};
    const Tensor out{g->out, g->ld_out, cols, "out"};
    for (const Tensor* t : {&ins[0], &ins[1], &ins[2], &out})
      if ((rc = check_tensor(*t))) return rc;
    if (nothing_to_do(*g, kZeroResults)) return MUONH_OK;
    for (const Tensor* t : {&ins[0], &ins[1], &ins[2], &out})
      if ((rc = check_address(*t))) return rc;
    if (!g->lse || !g->cu_seqlens) return fail(MUONH_EINVAL, "null pointer: lse or cu_seqlens");
    if (!aligned(g->lse, 4) || !aligned(g->cu_seqlens, 4)) return fail(MUONH_EINVAL, "misaligned lse or cu_seqlens");
    const Span lse{g->lse, (int64_t)row_bytes(*g)}, cu{g->cu_seqlens, (g->sequences + 1) * 4};
    if ((rc = check_sharing(&out, 1, ins, 3, g->tokens, {lse}, {cu}))) return rc;
    forget_older_errors();
    return launched(launch_attention_forward(device_args(*g, kZeroResults), reinterpret_cast<hipStream_t>(stream)), "attention_forward");
  });
}

int muonh_attention_backward_workspace(const muonh_attention_args* g, size_t* bytes) {
  return guarded([&]() -> int {
    if (!g || !bytes) return fail(MUONH_EINVAL, "null argument");
    int rc;
    if ((rc = check_shape(*g))) return rc;
    *bytes = workspace_of(*g);
    return MUONH_OK;
  });
}

int muonh_attention_backward(const muonh_attention_grad_args* b, void* stream) {
  return guarded([&]() -> int {
    if (!b) return fail(MUONH_EINVAL, "null argument");
    const muonh_attention_args* g = &b->a;
    int rc;
    if ((rc = check_shape(*g))) return rc;
    const int64_t cols = (int64_t)g->heads * g->dim, kv_cols = (int64_t)g->kv_heads * g->dim;
    const Tensor ins[] = {{g->q, g->ld_q, cols, "q"},     {g->k, g->ld_k, kv_cols, "k"},     {g->v, g->ld_v, kv_cols, "v"},
                          {g->out, g->ld_out, cols, "out"}, {b->dout, b->ld_dout, cols, "dout"}};
    const Tensor outs[] = {{b->dq, b->ld_dq, cols, "dq"}, {b->dk, b->ld_dk, kv_cols, "dk"}, {b->dv, b->ld_dv, kv_cols, "dv"}};
    for (const Tensor& t : ins)
      if ((rc = check_tensor(t))) return rc;
    for (const Tensor& t : outs)
      if ((rc = check_tensor(t))) return rc;
    if (nothing_to_do(*g, kZeroGradients)) return MUONH_OK;
    for (const Tensor& t : ins)
      if ((rc = check_address(t))) return rc;
    for (const Tensor& t : outs)
      if ((rc = check_address(t))) return rc;
    if (!g->lse || !g->cu_seqlens) return fail(MUONH_EINVAL, "null pointer: lse or cu_seqlens");
    if (!aligned(g->lse, 4) || !aligned(g->cu_seqlens, 4)) return fail(MUONH_EINVAL, "misaligned lse or cu_seqlens");
    const size_t need = workspace_of(*g);
    if (need > 0 && (!b->workspace || b->workspace_bytes < need))
      return fail(MUONH_ENOMEM, "workspace too small: need " + std::to_string(need) + " bytes");
    if (!aligned(b->workspace, kAlign)) return fail(MUONH_EINVAL, "workspace must be 256-byte aligned");
    const Span lse{g->lse, (int64_t)row_bytes(*g)}, cu{g->cu_seqlens, (g->sequences + 1) * 4};
    const Span ws{b->workspace, (int64_t)need};
    if ((rc = check_sharing(outs, 3, ins, 5, g->tokens, {ws}, {lse, cu}))) return rc;
    AttentionGradArgs a{};
    a.a = device_args(*g, kZeroGradients);
    a.dout = static_cast<const uint16_t*>(b->dout);
    a.dq = static_cast<uint16_t*>(b->dq);
    a.dk = static_cast<uint16_t*>(b->dk);
    a.dv = static_cast<uint16_t*>(b->dv);
    a.lddo = b->ld_dout;
    a.lddq = b->ld_dq;
    a.lddk = b->ld_dk;
    a.lddv = b->ld_dv;
    a.row_lse = static_cast<float*>(b->workspace);
    a.row_delta = reinterpret_cast<float*>(static_cast<uint8_t*>(b->workspace) + need / 2);
    forget_older_errors();
    return launched(launch_attention_backward(a, reinterpret_cast<hipStream_t>(stream)), "attention_backward");
  });
}

}  // extern "C"
