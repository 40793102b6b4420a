// attention.cuh -- what the attention kernels share: the sequence that a token
// belongs to, and one row of each result computed by a warp from its definition.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

// First token and end (one past the last token) of the sequence that holds token i,
// or an empty range for a token past the last sequence.  Clamped around i, so that
// offsets that do not ascend cannot lead outside the tensors.
struct Span { int begin, end; };

__device__ __forceinline__ Span sequence_of(const AttentionLaunch& L, int i) {
  if (L.cu == nullptr) return {0, L.T};
  int lo = 0, hi = L.n_seqs;             // last s in [0, n_seqs] with cu[s] <= i
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(L.cu + mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  if (lo >= L.n_seqs) return {i + 1, i};
  return {min(max(__ldg(L.cu + lo), 0), i), min(max(__ldg(L.cu + lo + 1), i + 1), L.T)};
}

// ---- rows by definition -------------------------------------------------
// A lane holds the elements 2 lane, 2 lane + 1 of each 64-element half of a head.
struct Row { float v[4]; };

__device__ __forceinline__ Row load_row(const __nv_bfloat16* p, int dim) {
  const int lane = threadIdx.x & 31;
  Row r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 64 * h + 2 * lane;
    unsigned int x = 0;
    if (d < dim) x = *reinterpret_cast<const unsigned int*>(p + d);
    r.v[2 * h] = __uint_as_float(x << 16);
    r.v[2 * h + 1] = __uint_as_float(x & 0xffff0000u);
  }
  return r;
}

__device__ __forceinline__ float dot_row(const Row& a, const Row& b) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(a.v[j], b.v[j], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// acc += f x
__device__ __forceinline__ void axpy(Row& acc, float f, const Row& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc.v[j] = fmaf(f, x.v[j], acc.v[j]);
}

__device__ __forceinline__ void store_row(__nv_bfloat16* p, const Row& r, int dim) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 64 * h + 2 * lane;
    if (d < dim)
      *reinterpret_cast<__nv_bfloat162*>(p + d) =
          __floats2bfloat162_rn(r.v[2 * h], r.v[2 * h + 1]);
  }
}

// Output row i of query head h (and its log-sum-exp) over the keys begin..i.
__device__ __noinline__ Row out_row(const AttentionLaunch& L, int h, int i, int begin,
                                    float* lse) {
  const int kh = h / L.group;
  const Row q = load_row(L.q.row(i, h), L.dim);
  Row acc = {{0.f, 0.f, 0.f, 0.f}};
  float m = -INFINITY, l = 0.f;
  for (int j = begin; j <= i; ++j) {
    const float s = L.scale * dot_row(q, load_row(L.k.row(j, kh), L.dim));
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = __expf(m - base), p = __expf(s - base);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.v[e] *= f;
    axpy(acc, p, load_row(L.v.row(j, kh), L.dim));
    m = mn;
  }
  *lse = l == 0.f ? -INFINITY : m + logf(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.v[e] *= inv;
  return acc;
}

// Query gradient row i of head h.
__device__ __noinline__ Row dq_row(const AttentionLaunch& L, int h, int i, int begin) {
  const int kh = h / L.group;
  const Row q = load_row(L.q.row(i, h), L.dim);
  const Row g = load_row(L.dout.row(i, h), L.dim);
  const float delta = dot_row(g, load_row(L.o.row(i, h), L.dim));
  const float lse = L.lse[static_cast<size_t>(h) * L.T + i];
  Row acc = {{0.f, 0.f, 0.f, 0.f}};
  for (int j = begin; j <= i; ++j) {
    const Row k = load_row(L.k.row(j, kh), L.dim);
    const float p = __expf(L.scale * dot_row(q, k) - lse);
    axpy(acc, p * (dot_row(g, load_row(L.v.row(j, kh), L.dim)) - delta), k);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.v[e] *= L.scale;
  return acc;
}

// Key and value gradient rows j of key head kh, over the queries j..end-1 of its group.
__device__ __noinline__ void dkv_row(const AttentionLaunch& L, int kh, int j, int end, Row& dk,
                                     Row& dv) {
  const Row k = load_row(L.k.row(j, kh), L.dim);
  const Row v = load_row(L.v.row(j, kh), L.dim);
  dk = dv = {{0.f, 0.f, 0.f, 0.f}};
  for (int h = kh * L.group; h < (kh + 1) * L.group; ++h)
    for (int i = j; i < end; ++i) {
      const Row q = load_row(L.q.row(i, h), L.dim);
      const Row g = load_row(L.dout.row(i, h), L.dim);
      const float delta = dot_row(g, load_row(L.o.row(i, h), L.dim));
      const float lse = L.lse[static_cast<size_t>(h) * L.T + i];
      const float p = __expf(L.scale * dot_row(q, k) - lse);
      axpy(dv, p, g);
      axpy(dk, p * (dot_row(g, v) - delta), q);
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) dk.v[e] *= L.scale;
}

}  // namespace attn
}  // namespace muon
