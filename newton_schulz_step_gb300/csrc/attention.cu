// attention.cu -- causal attention over packed sequences with grouped key/value
// heads, and its gradients: one warp computes one row from the definition.
#include "attention.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads)
    attention_kernel(const __grid_constant__ AttentionLaunch L) {
  if (ptx::status_set(L.status)) return;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(L.T) * L.hq) return;
  const int i = static_cast<int>(w / L.hq), h = static_cast<int>(w % L.hq);
  float lse;
  const attn::Row r = attn::out_row(L, h, i, attn::sequence_of(L, i).begin, &lse);
  attn::store_row(L.out.row(i, h), r, L.dim);
  if ((threadIdx.x & 31) == 0) L.lse[static_cast<size_t>(h) * L.T + i] = lse;
}

__global__ void __launch_bounds__(kThreads)
    attention_dq_kernel(const __grid_constant__ AttentionLaunch L) {
  if (ptx::status_set(L.status)) return;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(L.T) * L.hq) return;
  const int i = static_cast<int>(w / L.hq), h = static_cast<int>(w % L.hq);
  attn::store_row(L.dq.row(i, h), attn::dq_row(L, h, i, attn::sequence_of(L, i).begin), L.dim);
}

__global__ void __launch_bounds__(kThreads)
    attention_dkv_kernel(const __grid_constant__ AttentionLaunch L) {
  if (ptx::status_set(L.status)) return;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(L.T) * L.hk) return;
  const int j = static_cast<int>(w / L.hk), kh = static_cast<int>(w % L.hk);
  attn::Row dk, dv;
  attn::dkv_row(L, kh, j, attn::sequence_of(L, j).end, dk, dv);
  attn::store_row(L.dk.row(j, kh), dk, L.dim);
  attn::store_row(L.dv.row(j, kh), dv, L.dim);
}

int blocks_for(long long rows) { return static_cast<int>((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_attention(const AttentionLaunch& l, cudaStream_t s) {
  attention_kernel<<<blocks_for(1ll * l.T * l.hq), kThreads, 0, s>>>(l);
  return cudaGetLastError();
}
cudaError_t launch_attention_dq(const AttentionLaunch& l, cudaStream_t s) {
  attention_dq_kernel<<<blocks_for(1ll * l.T * l.hq), kThreads, 0, s>>>(l);
  return cudaGetLastError();
}
cudaError_t launch_attention_dkv(const AttentionLaunch& l, cudaStream_t s) {
  attention_dkv_kernel<<<blocks_for(1ll * l.T * l.hk), kThreads, 0, s>>>(l);
  return cudaGetLastError();
}

}  // namespace muon
