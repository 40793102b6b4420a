// attention_api.cu -- host side of the attention path's entry points declared in
// include/muon_gb300.h: argument checks, workspace layout, launches.
//
// Everything is enqueued on the caller's stream; nothing here synchronises or
// allocates device memory.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "views.h"

using namespace muon;

namespace {

constexpr int kMaxHeads = 65535;

bool flag(int x) { return x == 0 || x == 1; }

// Checks a view of [tokens, heads, dim] elements of `size` bytes and, for a
// dimension of one entry, replaces its (unused) stride by a valid one.
bool view_ok(muon_heads* v, int tokens, int heads, int dim, int size) {
  if (!v->data || !aligned16(v->data)) return false;
  const long long unit = 16 / size;
  if (heads == 1) v->head_stride = dim;
  if (tokens == 1) v->token_stride = 1ll * heads * dim;
  constexpr long long kMaxStride = 1ll << 38;   // below 2^40 bytes (tensor maps)
  return v->head_stride > 0 && v->token_stride > 0 && v->head_stride < kMaxStride &&
         v->token_stride < kMaxStride && v->head_stride % unit == 0 &&
         v->token_stride % unit == 0;
}

// Rows of different (token, head) of an output do not overlap: one stride spans a
// row, the other all rows along the first.
bool rows_apart(const muon_heads& v, int tokens, int heads, int dim) {
  const long long lo = tokens == 1 ? v.head_stride
                       : heads == 1 ? v.token_stride
                                    : std::min(v.head_stride, v.token_stride);
  if (lo < dim) return false;
  if (tokens == 1 || heads == 1) return true;
  const bool head_inner = v.head_stride <= v.token_stride;
  return head_inner ? v.token_stride >= v.head_stride * (heads - 1) + dim
                    : v.head_stride >= v.token_stride * (tokens - 1) + dim;
}

template <typename T>
Heads<T> view(const muon_heads& v) {
  return {static_cast<T*>(v.data), v.token_stride, v.head_stride};
}

// ------------------------------------------------------------ norm and rotation
bool rope_dim_ok(int dim) { return dim >= 8 && dim <= kRopeMaxDim && dim % 8 == 0; }

size_t rope_workspace(int dim) {
  constexpr int kRows = kRopeMaxBlocks + 32;
  return kStatusBytes + (static_cast<size_t>(kRows) * 2 * dim * sizeof(float) + 255) / 256 * 256;
}

// Fills the launch from the spec and the views ([0] queries, [1] keys); dy is
// null for the forward pass.
muon_status rope_launch(NormRopeLaunch& L, const muon_norm_rope* s, muon_heads (&x)[2],
                        muon_heads (&y)[2], muon_heads* dy) {
  std::memset(&L, 0, sizeof(L));
  if (!s) return MUON_ERR_INVALID_ARG;
  if (s->dtype != MUON_F32 && s->dtype != MUON_BF16) return MUON_ERR_INVALID_ARG;
  if (s->tokens < 0 || s->q_heads < 0 || s->k_heads < 0 || s->q_heads > kMaxHeads ||
      s->k_heads > kMaxHeads || s->q_heads + s->k_heads == 0)
    return MUON_ERR_INVALID_ARG;
  if (1ll * s->tokens * (s->q_heads + s->k_heads) > INT_MAX - 65536) return MUON_ERR_UNSUPPORTED;
  if (!rope_dim_ok(s->head_dim) || s->rot_dim < 0 || s->rot_dim > s->head_dim ||
      s->rot_dim % 8 != 0)
    return MUON_ERR_INVALID_ARG;
  if (!flag(s->norm) || !flag(s->interleaved) || !std::isfinite(s->eps) || s->eps < 0.f)
    return MUON_ERR_INVALID_ARG;
  if (s->rot_dim > 0 && (s->table_len < 1 || !s->cos || !s->sin || !aligned16(s->cos) ||
                         !aligned16(s->sin)))
    return MUON_ERR_INVALID_ARG;
  // without positions, token t takes row t
  if (s->rot_dim > 0 && !s->positions && s->table_len < s->tokens) return MUON_ERR_INVALID_ARG;
  if (!s->norm && (s->q_weight || s->k_weight)) return MUON_ERR_INVALID_ARG;
  if ((s->q_weight && !aligned16(s->q_weight)) || (s->k_weight && !aligned16(s->k_weight)))
    return MUON_ERR_INVALID_ARG;
  const int size = s->dtype == MUON_BF16 ? 2 : 4;
  L.heads[0] = s->q_heads;
  L.heads[1] = s->k_heads;
  if (s->tokens > 0)
    for (int i = 0; i < 2; ++i) {
      if (L.heads[i] == 0) continue;
      const bool needs_x = !dy || s->norm;
      if (needs_x && !view_ok(&x[i], s->tokens, L.heads[i], s->head_dim, size))
        return MUON_ERR_INVALID_ARG;
      if (dy && !view_ok(&dy[i], s->tokens, L.heads[i], s->head_dim, size))
        return MUON_ERR_INVALID_ARG;
      if (!view_ok(&y[i], s->tokens, L.heads[i], s->head_dim, size) ||
          !rows_apart(y[i], s->tokens, L.heads[i], s->head_dim))
        return MUON_ERR_INVALID_ARG;
      L.x[i] = view<void>(x[i]);
      L.y[i] = view<void>(y[i]);
      if (dy) L.dy[i] = view<void>(dy[i]);
    }
  L.w[0] = s->q_weight;
  L.w[1] = s->k_weight;
  L.tokens = s->tokens;
  L.dim = s->head_dim;
  L.rot = s->rot_dim;
  L.norm = s->norm;
  L.interleaved = s->interleaved;
  L.bf16 = s->dtype == MUON_BF16;
  L.table_len = s->table_len;
  L.eps = s->eps;
  L.cos = s->cos;
  L.sin = s->sin;
  L.pos = s->positions;
  return MUON_OK;
}

// Outputs share no bytes with inputs or with each other, but a kind's output may be its own
// input: the lanes of a row have loaded it before they store it.
bool rope_apart(const NormRopeLaunch& L, const muon_heads (&x)[2], const muon_heads (&y)[2],
                const muon_heads* dy) {
  const int size = L.bf16 ? 2 : 4;
  auto rows = [&](const muon_heads& v, int i) {
    return rows_of(v, L.tokens, L.heads[i], L.dim, size);
  };
  for (int i = 0; i < 2; ++i) {
    if (L.heads[i] == 0) continue;
    const Rows out = rows(y[i], i);
    if (i == 1 && L.heads[0] > 0 && overlap(out, rows(y[0], 0))) return false;
    for (int j = 0; j < 2; ++j) {
      if (L.heads[j] == 0) continue;
      auto clash = [&](const muon_heads& v) {
        const Rows in = rows(v, j);
        return !(i == j && same_rows(out, in)) && overlap(out, in);
      };
      if (((!dy || L.norm) && clash(x[j])) || (dy && clash(dy[j]))) return false;
    }
  }
  return true;
}

double rope_bytes(const NormRopeLaunch& L, int passes) {
  return 1.0 * L.tokens * (L.heads[0] + L.heads[1]) * L.dim * (L.bf16 ? 2 : 4) * passes;
}

// ------------------------------------------------------------ attention
bool attention_shape_ok(int tokens, int hq, int hk, int dim) {
  return tokens >= 0 && hq >= 1 && hk >= 1 && hq <= kMaxHeads && hk <= kMaxHeads &&
         hq % hk == 0 && dim >= 8 && dim <= 128 && dim % 8 == 0 &&
         1ll * tokens * hq <= INT_MAX - 65536;
}

// Status block, then per query head and 128 tokens: 128 log-sum-exps, 128 deltas.
size_t attention_workspace(int tokens, int hq) {
  return kStatusBytes + static_cast<size_t>(hq) * ((tokens + 127) / 128) * 1024;
}

muon_status attention_launch(AttentionLaunch& L, const muon_attention_spec* s, void* ws,
                             size_t ws_bytes) {
  if (!s) return MUON_ERR_INVALID_ARG;
  if (!attention_shape_ok(s->tokens, s->q_heads, s->kv_heads, s->head_dim))
    return MUON_ERR_INVALID_ARG;
  if (s->n_seqs < 0 || (s->n_seqs > 0 && !s->cu_seqlens)) return MUON_ERR_INVALID_ARG;
  if (s->cu_seqlens && (reinterpret_cast<uintptr_t>(s->cu_seqlens) & 3u)) return MUON_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale) || s->scale <= 0.f) return MUON_ERR_INVALID_ARG;
  const muon_status st = check_workspace(ws, ws_bytes, attention_workspace(s->tokens, s->q_heads));
  if (st != MUON_OK) return st;
  std::memset(static_cast<void*>(&L), 0, sizeof(L));
  L.cu = s->cu_seqlens;
  L.n_seqs = s->n_seqs;
  L.T = s->tokens;
  L.hq = s->q_heads;
  L.hk = s->kv_heads;
  L.group = s->q_heads / s->kv_heads;
  L.dim = s->head_dim;
  L.scale = s->scale;
  L.status = static_cast<unsigned int*>(ws);
  return MUON_OK;
}

// Visible (query, key) pairs times heads if the tokens were one sequence: the
// lengths are on the device, so this is the upper bound that the trace records.
double pair_bound(const AttentionLaunch& L) { return 0.5 * L.T * (L.T + 1.0) * L.hq; }

}  // namespace

extern "C" {

muon_status muon_qk_norm_rope(const muon_norm_rope* spec, muon_heads q, muon_heads k,
                              muon_heads q_out, muon_heads k_out, void* stream) {
  try {
    NormRopeLaunch L;
    muon_heads x[2] = {q, k}, y[2] = {q_out, k_out};
    const muon_status s = rope_launch(L, spec, x, y, nullptr);
    if (s != MUON_OK) return s;
    if (L.tokens == 0) return MUON_OK;
    int sms = 0;
    const muon_status ds = device_sms(&sms);
    if (ds != MUON_OK) return ds;
    if (!rope_apart(L, x, y, nullptr)) return MUON_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = counted_launch(st, MUON_K_NORM_ROPE, 0.0, rope_bytes(L, 2),
                                         [&] { return launch_norm_rope(L, false, sms, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

size_t muon_norm_rope_workspace_bytes(int head_dim) {
  return rope_dim_ok(head_dim) ? rope_workspace(head_dim) : 0;
}

muon_status muon_qk_norm_rope_backward(const muon_norm_rope* spec, muon_heads dq_out,
                                       muon_heads dk_out, muon_heads q, muon_heads k,
                                       muon_heads dq, muon_heads dk, float* dq_weight,
                                       float* dk_weight, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  try {
    NormRopeLaunch L;
    muon_heads x[2] = {q, k}, y[2] = {dq, dk}, dy[2] = {dq_out, dk_out};
    muon_status s = rope_launch(L, spec, x, y, dy);
    if (s != MUON_OK) return s;
    if ((L.w[0] != nullptr) != (dq_weight != nullptr) ||
        (L.w[1] != nullptr) != (dk_weight != nullptr))
      return MUON_ERR_INVALID_ARG;
    s = check_workspace(workspace, workspace_bytes, rope_workspace(L.dim));
    if (s != MUON_OK) return s;
    if (L.tokens == 0 && !dq_weight && !dk_weight) return MUON_OK;
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (L.tokens == 0) {                       // sums over nothing
      float* dw[2] = {dq_weight, dk_weight};
      for (float* p : dw)
        if (p && cudaMemsetAsync(p, 0, L.dim * sizeof(float), st) != cudaSuccess)
          return MUON_ERR_CUDA;
      return MUON_OK;
    }
    if (!rope_apart(L, x, y, dy)) return MUON_ERR_INVALID_ARG;
    L.dw[0] = dq_weight;
    L.dw[1] = dk_weight;
    L.status = static_cast<const unsigned int*>(workspace);
    L.ticket = static_cast<unsigned int*>(workspace) + 16;
    L.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    const WorkspaceTurn turn(workspace);
    const cudaError_t e =
        counted_launch(st, MUON_K_NORM_ROPE_BWD, 0.0, rope_bytes(L, L.norm ? 3 : 2),
                       [&] { return launch_norm_rope(L, true, sms, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

size_t muon_attention_workspace_bytes(int tokens, int q_heads, int kv_heads, int head_dim) {
  if (!attention_shape_ok(tokens, q_heads, kv_heads, head_dim)) return 0;
  return attention_workspace(tokens, q_heads);
}

muon_status muon_attention(const muon_attention_spec* spec, muon_heads q, muon_heads k,
                           muon_heads v, muon_heads out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  try {
    AttentionLaunch L;
    muon_status s = attention_launch(L, spec, workspace, workspace_bytes);
    if (s != MUON_OK) return s;
    if (L.T == 0) return MUON_OK;
    if (!view_ok(&q, L.T, L.hq, L.dim, 2) || !view_ok(&k, L.T, L.hk, L.dim, 2) ||
        !view_ok(&v, L.T, L.hk, L.dim, 2) || !view_ok(&out, L.T, L.hq, L.dim, 2) ||
        !rows_apart(out, L.T, L.hq, L.dim) || !lse || !aligned16(lse))
      return MUON_ERR_INVALID_ARG;
    auto of_q = [&](const muon_heads& x) { return rows_of(x, L.T, L.hq, L.dim, 2); };
    auto of_k = [&](const muon_heads& x) { return rows_of(x, L.T, L.hk, L.dim, 2); };
    if (!apart({of_q(out), rows_of(lse, 1ll * L.hq * L.T)}, {of_q(q), of_k(k), of_k(v)}))
      return MUON_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    L.q = view<const __nv_bfloat16>(q);
    L.k = view<const __nv_bfloat16>(k);
    L.v = view<const __nv_bfloat16>(v);
    L.out = view<__nv_bfloat16>(out);
    L.lse = lse;
    AttentionMaps M;
    if (!heads_tmap(&M.q, q, L.T, L.hq, L.dim) || !heads_tmap(&M.k, k, L.T, L.hk, L.dim) ||
        !heads_tmap(&M.v, v, L.T, L.hk, L.dim) || !heads_tmap(&M.out, out, L.T, L.hq, L.dim))
      return MUON_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const double heads = 2.0 * L.T * (2.0 * L.hq + 2.0 * L.hk) * L.dim;
    const cudaError_t e =
        counted_launch(st, MUON_K_ATTENTION, 4.0 * L.dim * pair_bound(L), heads,
                       [&] { return launch_attention(M, L, sms, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

muon_status muon_attention_backward(const muon_attention_spec* spec, muon_heads dout,
                                    muon_heads q, muon_heads k, muon_heads v, muon_heads out,
                                    const float* lse, muon_heads dq, muon_heads dk,
                                    muon_heads dv, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  try {
    AttentionLaunch L;
    muon_status s = attention_launch(L, spec, workspace, workspace_bytes);
    if (s != MUON_OK) return s;
    if (L.T == 0) return MUON_OK;
    muon_heads* q_views[] = {&dout, &q, &out, &dq};
    muon_heads* k_views[] = {&k, &v, &dk, &dv};
    for (muon_heads* x : q_views)
      if (!view_ok(x, L.T, L.hq, L.dim, 2)) return MUON_ERR_INVALID_ARG;
    for (muon_heads* x : k_views)
      if (!view_ok(x, L.T, L.hk, L.dim, 2)) return MUON_ERR_INVALID_ARG;
    if (!rows_apart(dq, L.T, L.hq, L.dim) || !rows_apart(dk, L.T, L.hk, L.dim) ||
        !rows_apart(dv, L.T, L.hk, L.dim) || !lse || !aligned16(lse))
      return MUON_ERR_INVALID_ARG;
    // (the second launch reads q, k, v and dout again, after the first has written dq)
    auto of_q = [&](const muon_heads& x) { return rows_of(x, L.T, L.hq, L.dim, 2); };
    auto of_k = [&](const muon_heads& x) { return rows_of(x, L.T, L.hk, L.dim, 2); };
    if (!apart({of_q(dq), of_k(dk), of_k(dv)},
               {of_q(dout), of_q(q), of_k(k), of_k(v), of_q(out), rows_of(lse, 1ll * L.hq * L.T)}))
      return MUON_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    L.q = view<const __nv_bfloat16>(q);
    L.k = view<const __nv_bfloat16>(k);
    L.v = view<const __nv_bfloat16>(v);
    L.o = view<const __nv_bfloat16>(out);
    L.dout = view<const __nv_bfloat16>(dout);
    L.dq = view<__nv_bfloat16>(dq);
    L.dk = view<__nv_bfloat16>(dk);
    L.dv = view<__nv_bfloat16>(dv);
    L.lse = const_cast<float*>(lse);
    L.stats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    AttentionMaps M;
    if (!heads_tmap(&M.q, q, L.T, L.hq, L.dim) || !heads_tmap(&M.k, k, L.T, L.hk, L.dim) ||
        !heads_tmap(&M.v, v, L.T, L.hk, L.dim) || !heads_tmap(&M.dout, dout, L.T, L.hq, L.dim) ||
        !heads_tmap(&M.dq, dq, L.T, L.hq, L.dim) || !heads_tmap(&M.dk, dk, L.T, L.hk, L.dim) ||
        !heads_tmap(&M.dv, dv, L.T, L.hk, L.dim))
      return MUON_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const double row = 2.0 * L.T * L.dim;
    // (dk, dv reads what dq leaves in the workspace)
    const WorkspaceTurn turn(workspace);
    cudaError_t e = counted_launch(
        st, MUON_K_ATTENTION_DQ, 6.0 * L.dim * pair_bound(L), row * (4.0 * L.hq + 2.0 * L.hk),
        [&] { return launch_attention_dq(M, L, st); });
    if (e != cudaSuccess) return MUON_ERR_CUDA;
    e = counted_launch(st, MUON_K_ATTENTION_DKV, 8.0 * L.dim * pair_bound(L),
                       row * (2.0 * L.hq + 4.0 * L.hk),
                       [&] { return launch_attention_dkv(M, L, sms, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

}  // extern "C"
