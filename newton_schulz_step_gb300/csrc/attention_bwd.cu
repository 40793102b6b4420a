// attention_bwd.cu -- gradients of causal attention over packed sequences with grouped
// key/value heads: one warp computes one row from the definition.
#include "attention.cuh"

namespace muon {
namespace {

constexpr int kRowThreads = 256;
constexpr int kWarps = kRowThreads / 32;

__device__ __forceinline__ void store_row(__nv_bfloat16* p, const attn::Row& r, int dim) {
  const int lane = threadIdx.x & 31;
  for (int h = 0; h < 2; ++h)
    if (64 * h + 2 * lane < dim)
      *reinterpret_cast<uint32_t*>(p + 64 * h + 2 * lane) =
          attn::pack2(r.v[2 * h], r.v[2 * h + 1]);
}

__global__ void __launch_bounds__(kRowThreads)
    attention_dq_kernel(const __grid_constant__ AttentionLaunch L) {
  if (ptx::status_set(L.status)) return;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(L.T) * L.hq) return;
  const int i = static_cast<int>(w / L.hq), h = static_cast<int>(w % L.hq);
  store_row(L.dq.row(i, h), attn::dq_row(L, h, i, attn::sequence_of(L, i).begin), L.dim);
}

__global__ void __launch_bounds__(kRowThreads)
    attention_dkv_kernel(const __grid_constant__ AttentionLaunch L) {
  if (ptx::status_set(L.status)) return;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(L.T) * L.hk) return;
  const int j = static_cast<int>(w / L.hk), kh = static_cast<int>(w % L.hk);
  attn::Row dk, dv;
  attn::dkv_row(L, kh, j, attn::sequence_of(L, j).end, dk, dv);
  store_row(L.dk.row(j, kh), dk, L.dim);
  store_row(L.dv.row(j, kh), dv, L.dim);
}

int blocks_for(long long rows) { return static_cast<int>((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_attention_dq(const AttentionLaunch& l, cudaStream_t s) {
  attention_dq_kernel<<<blocks_for(1ll * l.T * l.hq), kRowThreads, 0, s>>>(l);
  return cudaGetLastError();
}
cudaError_t launch_attention_dkv(const AttentionLaunch& l, cudaStream_t s) {
  attention_dkv_kernel<<<blocks_for(1ll * l.T * l.hk), kRowThreads, 0, s>>>(l);
  return cudaGetLastError();
}

}  // namespace muon
