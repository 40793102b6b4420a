// block_api.cu -- host side of the RMS norm, the embedding and the gradients' clipping
// declared in include/muon_gb300.h: argument checks, workspace layout, launches.
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

constexpr int kMaxTokens = INT_MAX - 65536;
constexpr int kMaxRows = 1 << 30;
constexpr int kMaxEmbeddingDim = 65536;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool dtype_ok(int t) { return t == MUON_F32 || t == MUON_BF16; }
int size_of(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }

// Checks a view of [rows, cols] elements of `size` bytes (cols a multiple of 8); rows of a
// view of bytes are 8-byte aligned, others 16.
bool matrix_ok(muon_matrix* v, int rows, int cols, int size) {
  if (!v->data || !aligned16(v->data)) return false;
  if (rows == 1) v->row_stride = cols;
  constexpr long long kMaxStride = 1ll << 38;
  return v->row_stride >= cols && v->row_stride < kMaxStride &&
         v->row_stride % (size == 1 ? 8 : 16 / size) == 0;
}
Rows rows_of(const muon_matrix& v, int rows, int cols, int size) {
  return {reinterpret_cast<uintptr_t>(v.data), v.row_stride * size, 0, 1ll * cols * size, rows, 1};
}
Rows flat(const void* p, long long bytes) {
  return {reinterpret_cast<uintptr_t>(p), 0, 0, bytes, 1, 1};
}

// ------------------------------------------------------------ RMS norm
bool norm_dim_ok(int dim) { return dim >= 8 && dim <= kRmsNormMaxDim && dim % 8 == 0; }
size_t norm_workspace(int dim) {
  return kStatusBytes + align256(static_cast<size_t>(kRmsNormMaxBlocks) * dim * sizeof(float));
}
bool norm_spec_ok(const muon_rms_norm_spec* s) {
  return s && dtype_ok(s->dtype) && s->tokens >= 0 && s->tokens <= kMaxTokens &&
         norm_dim_ok(s->dim) && std::isfinite(s->eps) && s->eps >= 0.f && aligned16(s->weight);
}

// muon_rms_norm (scales == NULL) and muon_rms_norm_fp8.
muon_status norm_forward(const muon_rms_norm_spec* s, bool eight_bits, int group, muon_matrix x,
                         muon_matrix residual, muon_matrix out, float* scales, muon_matrix sum,
                         void* stream) {
  if (!norm_spec_ok(s) || (group != 0 && group != 128)) return MUON_ERR_INVALID_ARG;
  const int t = s->tokens, d = s->dim, size = size_of(s->dtype), out_size = eight_bits ? 1 : size;
  const bool has_res = residual.data != nullptr;
  if (has_res != (sum.data != nullptr) && t > 0) return MUON_ERR_INVALID_ARG;
  if (t == 0) return MUON_OK;
  if (!matrix_ok(&x, t, d, size) || !matrix_ok(&out, t, d, out_size) ||
      (has_res && (!matrix_ok(&residual, t, d, size) || !matrix_ok(&sum, t, d, size))))
    return MUON_ERR_INVALID_ARG;
  if (eight_bits && (!scales || (reinterpret_cast<uintptr_t>(scales) & 3u)))
    return MUON_ERR_INVALID_ARG;
  const int groups = group == 0 ? 1 : (d + group - 1) / group;
  // a row is loaded whole before any of it is stored: an output in the inputs' type may be the
  // very view of an input, and shares bytes with nothing else
  const Rows r_x = rows_of(x, t, d, size), r_out = rows_of(out, t, d, out_size);
  const Rows r_w = flat(s->weight, 4ll * d), r_s = flat(scales, 4ll * t * groups);
  const Rows r_res = has_res ? rows_of(residual, t, d, size) : r_x;
  auto clash = [&](const Rows& o, bool may_be) {
    for (const Rows& in : {r_x, r_res})
      if (!(may_be && same_rows(o, in)) && overlap(o, in)) return true;
    return s->weight && overlap(o, r_w);
  };
  if (clash(r_out, !eight_bits)) return MUON_ERR_INVALID_ARG;
  if (has_res) {
    const Rows r_sum = rows_of(sum, t, d, size);
    if (clash(r_sum, true) || overlap(r_sum, r_out) || (eight_bits && overlap(r_sum, r_s)))
      return MUON_ERR_INVALID_ARG;
  }
  if (eight_bits && (clash(r_s, false) || overlap(r_s, r_out))) return MUON_ERR_INVALID_ARG;
  int sms = 0;
  const muon_status ds = device_sms(&sms);
  if (ds != MUON_OK) return ds;
  RmsNormLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.x = x.data;
  L.res = residual.data;
  L.y = out.data;
  L.sum = sum.data;
  L.w = s->weight;
  L.scales = scales;
  L.x_stride = x.row_stride;
  L.res_stride = residual.row_stride;
  L.y_stride = out.row_stride;
  L.sum_stride = sum.row_stride;
  L.tokens = t;
  L.dim = d;
  L.group = group;
  L.groups = groups;
  L.eps = s->eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const double bytes = 1.0 * t * d * (size * (has_res ? 3.0 : 1.0) + out_size);
  const cudaError_t e = counted_launch(st, MUON_K_RMS_NORM, 0.0, bytes, [&] {
    return launch_rms_norm(L, s->dtype == MUON_BF16, eight_bits, sms, st);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

// ------------------------------------------------------------ embedding
bool embedding_sizes_ok(int tokens, int dim) {
  return tokens >= 0 && tokens <= kMaxTokens && dim >= 8 && dim <= kMaxEmbeddingDim &&
         dim % 8 == 0;
}
bool embedding_spec_ok(const muon_embedding_spec* s) {
  return s && embedding_sizes_ok(s->tokens, s->dim) && s->rows >= 1 && s->rows <= kMaxRows &&
         (s->id_bytes == 4 || s->id_bytes == 8) && std::isfinite(s->scale) &&
         (s->tokens == 0 ||
          (s->ids && (reinterpret_cast<uintptr_t>(s->ids) & (s->id_bytes - 1)) == 0));
}
// Status block, number of sorted tokens, sorted and unsorted ids and tokens, pieces of runs.
size_t embedding_workspace(int tokens, int dim) {
  return kStatusBytes + 256 + 4 * align256(static_cast<size_t>(tokens) * 4) +
         align256(embedding_parts(tokens, dim) * sizeof(float));
}
void fill_embedding(EmbeddingLaunch& L, const muon_embedding_spec* s) {
  std::memset(&L, 0, sizeof(L));
  L.ids = s->ids;
  L.wide = s->id_bytes == 8;
  L.tokens = s->tokens;
  L.rows = s->rows;
  L.dim = s->dim;
  L.scale = s->scale;
}

}  // namespace

extern "C" {

muon_status muon_rms_norm(const muon_rms_norm_spec* spec, muon_matrix x, muon_matrix residual,
                          muon_matrix out, muon_matrix sum, void* stream) {
  try {
    return norm_forward(spec, false, 0, x, residual, out, nullptr, sum, stream);
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

muon_status muon_rms_norm_fp8(const muon_rms_norm_spec* spec, int group, muon_matrix x,
                              muon_matrix residual, muon_matrix out, float* scales,
                              muon_matrix sum, void* stream) {
  try {
    return norm_forward(spec, true, group, x, residual, out, scales, sum, stream);
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

size_t muon_rms_norm_workspace_bytes(int dim) { return norm_dim_ok(dim) ? norm_workspace(dim) : 0; }

muon_status muon_rms_norm_backward(const muon_rms_norm_spec* spec, muon_matrix dout,
                                   muon_matrix sum, muon_matrix dresidual, muon_matrix dx,
                                   float* dweight, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  try {
    if (!norm_spec_ok(spec)) return MUON_ERR_INVALID_ARG;
    const int t = spec->tokens, d = spec->dim, size = size_of(spec->dtype);
    const bool has_res = dresidual.data != nullptr;
    if ((spec->weight != nullptr) != (dweight != nullptr) || !aligned16(dweight))
      return MUON_ERR_INVALID_ARG;
    muon_status s = check_workspace(workspace, workspace_bytes, norm_workspace(d));
    if (s != MUON_OK) return s;
    if (t == 0 && !dweight) return MUON_OK;
    if (t > 0) {
      if (!matrix_ok(&dout, t, d, size) || !matrix_ok(&sum, t, d, size) ||
          !matrix_ok(&dx, t, d, size) || (has_res && !matrix_ok(&dresidual, t, d, size)))
        return MUON_ERR_INVALID_ARG;
      const Rows r_dx = rows_of(dx, t, d, size);
      const Rows ins[3] = {rows_of(dout, t, d, size), rows_of(sum, t, d, size),
                           has_res ? rows_of(dresidual, t, d, size) : rows_of(dout, t, d, size)};
      const Rows r_w = flat(spec->weight, 4ll * d), r_dw = flat(dweight, 4ll * d);
      for (const Rows& in : ins) {
        if (!same_rows(r_dx, in) && overlap(r_dx, in)) return MUON_ERR_INVALID_ARG;
        if (dweight && overlap(r_dw, in)) return MUON_ERR_INVALID_ARG;
      }
      if (dweight && (overlap(r_dw, r_w) || overlap(r_dw, r_dx) || overlap(r_dx, r_w)))
        return MUON_ERR_INVALID_ARG;
    }
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (t == 0)                                // a sum over nothing
      return cudaMemsetAsync(dweight, 0, d * sizeof(float), st) == cudaSuccess ? MUON_OK
                                                                             : MUON_ERR_CUDA;
    RmsNormLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.x = sum.data;
    L.dy = dout.data;
    L.res = dresidual.data;
    L.y = dx.data;
    L.w = spec->weight;
    L.x_stride = sum.row_stride;
    L.dy_stride = dout.row_stride;
    L.res_stride = dresidual.row_stride;
    L.y_stride = dx.row_stride;
    L.tokens = t;
    L.dim = d;
    L.eps = spec->eps;
    L.status = static_cast<const unsigned int*>(workspace);
    if (dweight)
      L.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    const WorkspaceTurn turn(dweight ? workspace : nullptr);
    cudaError_t e = counted_launch(
        st, MUON_K_RMS_NORM_BWD, 0.0, 1.0 * t * d * size * (has_res ? 4.0 : 3.0),
        [&] { return launch_rms_norm_backward(L, spec->dtype == MUON_BF16, st); });
    if (e == cudaSuccess && dweight)
      e = counted_launch(st, MUON_K_RMS_NORM_WEIGHT, 0.0,
                         4.0 * rms_norm_blocks(t, d) * d,
                         [&] { return launch_rms_norm_weight(L, dweight, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

muon_status muon_embedding(const muon_embedding_spec* spec, int table_dtype, muon_matrix table,
                           int out_dtype, muon_matrix out, void* stream) {
  try {
    if (!embedding_spec_ok(spec) || !dtype_ok(table_dtype) || !dtype_ok(out_dtype))
      return MUON_ERR_INVALID_ARG;
    const int t = spec->tokens, d = spec->dim;
    if (t == 0) return MUON_OK;
    if (!matrix_ok(&table, spec->rows, d, size_of(table_dtype)) ||
        !matrix_ok(&out, t, d, size_of(out_dtype)))
      return MUON_ERR_INVALID_ARG;
    const Rows r_out = rows_of(out, t, d, size_of(out_dtype));
    if (overlap(r_out, rows_of(table, spec->rows, d, size_of(table_dtype))) ||
        overlap(r_out, flat(spec->ids, 1ll * t * spec->id_bytes)))
      return MUON_ERR_INVALID_ARG;
    int sms = 0;
    const muon_status s = device_sms(&sms);
    if (s != MUON_OK) return s;
    EmbeddingLaunch L;
    fill_embedding(L, spec);
    L.table = table.data;
    L.table_stride = table.row_stride;
    L.out = out.data;
    L.out_stride = out.row_stride;
    L.out_bf16 = out_dtype == MUON_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = counted_launch(
        st, MUON_K_EMBEDDING, 0.0, 1.0 * t * d * (size_of(table_dtype) + size_of(out_dtype)),
        [&] { return launch_embedding(L, table_dtype == MUON_BF16, sms, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

size_t muon_embedding_workspace_bytes(int tokens, int dim) {
  return embedding_sizes_ok(tokens, dim) ? embedding_workspace(tokens, dim) : 0;
}

muon_status muon_embedding_backward(const muon_embedding_spec* spec, int dout_dtype,
                                    muon_matrix dout, int dtable_dtype, muon_matrix dtable,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!embedding_spec_ok(spec) || !dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype))
      return MUON_ERR_INVALID_ARG;
    const int t = spec->tokens, d = spec->dim, size = size_of(dtable_dtype);
    muon_status s = check_workspace(workspace, workspace_bytes, embedding_workspace(t, d));
    if (s != MUON_OK) return s;
    if (!matrix_ok(&dtable, spec->rows, d, size)) return MUON_ERR_INVALID_ARG;
    if (t > 0) {
      if (!matrix_ok(&dout, t, d, size_of(dout_dtype))) return MUON_ERR_INVALID_ARG;
      const Rows r_dt = rows_of(dtable, spec->rows, d, size);
      if (overlap(r_dt, rows_of(dout, t, d, size_of(dout_dtype))) ||
          overlap(r_dt, flat(spec->ids, 1ll * t * spec->id_bytes)))
        return MUON_ERR_INVALID_ARG;
    }
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (t == 0)                                // sums over nothing
      return cudaMemset2DAsync(dtable.data, dtable.row_stride * size, 0, 1ll * d * size,
                               spec->rows, st) == cudaSuccess
                 ? MUON_OK
                 : MUON_ERR_CUDA;
    EmbeddingLaunch L;
    fill_embedding(L, spec);
    L.dout = dout.data;
    L.dout_stride = dout.row_stride;
    L.out = dtable.data;
    L.out_stride = dtable.row_stride;
    L.out_bf16 = dtable_dtype == MUON_BF16;
    L.status = static_cast<const unsigned int*>(workspace);
    uint8_t* p = static_cast<uint8_t*>(workspace) + kStatusBytes;
    L.count = reinterpret_cast<uint32_t*>(p);
    p += 256;
    const size_t list = align256(static_cast<size_t>(t) * 4);
    for (int i = 0; i < 2; ++i) {
      L.keys[i] = reinterpret_cast<uint32_t*>(p);
      L.order[i] = reinterpret_cast<uint32_t*>(p + list);
      p += 2 * list;
    }
    L.parts = reinterpret_cast<float*>(p);
    const WorkspaceTurn turn(workspace);
    cudaError_t e = counted_launch(st, MUON_K_EMBEDDING_SORT, 0.0,
                                   1.0 * spec->rows * d * size + 16.0 * t,
                                   [&] { return launch_embedding_sort(L, sms, st); });
    if (e == cudaSuccess)
      e = counted_launch(st, MUON_K_EMBEDDING_SUM, 0.0, 1.0 * t * d * size_of(dout_dtype),
                         [&] { return launch_embedding_sum(L, dout_dtype == MUON_BF16, st); });
    if (e == cudaSuccess && embedding_parts(t, d) > 0)
      e = counted_launch(st, MUON_K_EMBEDDING_JOIN, 0.0, 0.0,
                         [&] { return launch_embedding_join(L, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

size_t muon_clip_workspace_bytes(int n_tensors) {
  if (n_tensors < 0) return 0;
  const size_t launches = (static_cast<size_t>(n_tensors) + kMaxClipTensors - 1) / kMaxClipTensors;
  return kStatusBytes + align256(std::max<size_t>(1, launches) * kClipBlocks * sizeof(float2));
}

muon_status muon_clip_grad_norm(const muon_grad_tensor* tensors, int n_tensors, float max_norm,
                                float eps, float* norm, void* workspace, size_t workspace_bytes,
                                void* stream) {
  try {
    if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !norm ||
        (reinterpret_cast<uintptr_t>(norm) & 3u) || !(max_norm >= 0.f) || !std::isfinite(eps) ||
        eps < 0.f)
      return MUON_ERR_INVALID_ARG;
    // an infinite max_norm leaves the gradients as they are, but copies to other outputs
    const bool clip = std::isfinite(max_norm) ||
                      std::any_of(tensors, tensors + n_tensors, [](const muon_grad_tensor& T) {
                        return T.numel > 0 && T.out &&
                               (T.out != T.grad || T.out_dtype != T.g_dtype);
                      });
    const Rows r_norm = flat(norm, sizeof(float));
    bool in_place = true;
    for (int i = 0; i < n_tensors; ++i) {
      const muon_grad_tensor& T = tensors[i];
      if (T.numel < 0 || !dtype_ok(T.g_dtype)) return MUON_ERR_INVALID_ARG;
      if (T.numel == 0) continue;
      if (!T.grad || !aligned16(T.grad) || overlap(r_norm, flat(T.grad, T.numel * size_of(T.g_dtype))))
        return MUON_ERR_INVALID_ARG;
      if (!clip) continue;
      if (!T.out || !aligned16(T.out) || !dtype_ok(T.out_dtype) ||
          overlap(r_norm, flat(T.out, T.numel * size_of(T.out_dtype))))
        return MUON_ERR_INVALID_ARG;
      const bool same = T.out == T.grad && T.out_dtype == T.g_dtype;
      if (!same && overlap(flat(T.out, T.numel * size_of(T.out_dtype)),
                           flat(T.grad, T.numel * size_of(T.g_dtype))))
        return MUON_ERR_INVALID_ARG;
      in_place &= same;
    }
    muon_status s = check_workspace(workspace, workspace_bytes, muon_clip_workspace_bytes(n_tensors));
    if (s != MUON_OK) return s;
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    ClipLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.parts = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    L.status = static_cast<const unsigned int*>(workspace);
    L.max_norm = max_norm;
    L.eps = eps;
    L.in_place = in_place;
    // the tensors of one launch, from the i-th on; how many of the list it covers
    double bytes_in = 0.0, bytes_out = 0.0;
    auto fill = [&](int i) {
      L.n_tensors = 0;
      L.total_units = 0;
      bytes_in = bytes_out = 0.0;
      int j = i;
      for (; j < n_tensors && L.n_tensors < kMaxClipTensors; ++j) {
        const muon_grad_tensor& T = tensors[j];
        if (T.numel == 0) continue;
        ClipTensor& c = L.t[L.n_tensors++];
        c.g = T.grad;
        c.out = T.out;
        c.n = T.numel;
        c.unit_begin = L.total_units;
        c.g_bf16 = T.g_dtype == MUON_BF16;
        c.out_bf16 = T.out_dtype == MUON_BF16;
        L.total_units += (T.numel + kClipUnit - 1) / kClipUnit;
        bytes_in += 1.0 * T.numel * size_of(T.g_dtype);
        bytes_out += 1.0 * T.numel * (c.out_bf16 ? 2 : 4);
      }
      return j;
    };
    const WorkspaceTurn turn(workspace);
    cudaError_t e = cudaSuccess;
    int i = 0, launches = 0;
    do {
      i = fill(i);
      const int blocks = clip_blocks(L, sms);
      e = counted_launch(st, MUON_K_GRAD_SQUARES, 0.0, bytes_in,
                         [&] { return launch_grad_squares(L, blocks, st); });
      L.part_begin += blocks;
      ++launches;
    } while (e == cudaSuccess && i < n_tensors);
    L.n_parts = L.part_begin;
    // (with one launch its tensors are still in place)
    i = 0;
    L.norm = norm;
    do {
      if (!clip) {
        L.total_units = 0;
        i = n_tensors;
      } else {
        i = launches > 1 ? fill(i) : n_tensors;
      }
      if (e == cudaSuccess)
        e = counted_launch(st, MUON_K_CLIP, 0.0, clip ? bytes_in + bytes_out : 0.0,
                           [&] { return launch_clip(L, sms, st); });
      L.norm = nullptr;
    } while (e == cudaSuccess && i < n_tensors);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

}  // extern "C"
