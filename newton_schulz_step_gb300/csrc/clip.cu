// clip.cu -- the norm of all gradients of a model together, and the gradients clipped by it:
//
//   norm = (sum over all tensors and elements of g^2)^1/2
//   out  = g c,  c = min(1, max_norm / (norm + eps))
//
// Two passes over the gradients, both bound by HBM: squares summed into one part a block,
// then the factor (every block adds the few hundred parts, in order) and the products.  The
// second pass walks the gradients backwards: it starts with what the first read last and L2
// still holds, and its own stores are marked to leave L2 first.  Gradients of up to about
// 100 MB are read from HBM once that way.
//
// Squares are taken and added in fp32 a thread (a magnitude from 2^64 on makes the norm
// infinite, one below 2^-75 adds nothing), the threads' sums are added in fp64.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kClipUnit / 8 / kThreads;      // vectors of 8 a thread and unit

struct Raw {
  uint4 a, b;                                        // b: fp32 only
};
__device__ __forceinline__ void load(const ClipTensor& T, long long e, Raw& r) {
  if (T.g_bf16) {
    r.a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(T.g) + e));
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(T.g) + e);
    r.a = __ldcg(p);
    r.b = __ldcg(p + 1);
  }
}
__device__ __forceinline__ void get(const ClipTensor& T, const Raw& r, float (&v)[8]) {
  const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (T.g_bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  } else {
    const uint32_t b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}
__device__ __forceinline__ float value(const ClipTensor& T, long long e) {
  return T.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(T.g)[e])
                  : static_cast<const float*>(T.g)[e];
}
__device__ __forceinline__ void store(const ClipTensor& T, long long e, const float (&v)[8]) {
  if (T.out_bf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(T.out) + e),
           make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(T.out) + e);
    __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
}

// Tensor of unit u: the last one that begins at or before it.
__device__ __forceinline__ const ClipTensor& tensor_of(const ClipLaunch& L, long long u) {
  int lo = 0, hi = L.n_tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.t[mid].unit_begin <= u) lo = mid;
    else hi = mid - 1;
  }
  return L.t[lo];
}

// Sum over the block, the same for every thread and run.
__device__ __forceinline__ double block_sum(double x, double* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) x += s[k];
  return x;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ ClipLaunch L) {
  __shared__ double s_sum[kThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
  for (long long u = blockIdx.x; u < L.total_units; u += gridDim.x) {
    const ClipTensor& T = tensor_of(L, u);
    const long long base = (u - T.unit_begin) * kClipUnit;
    if (base + kClipUnit <= T.n) {
      Raw r[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) load(T, base + 8ll * (i * kThreads + threadIdx.x), r[i]);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        float v[8];
        get(T, r[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(v[j], v[j], sum[j]);
      }
    } else {
      for (int i = 0; i < kVecs; ++i) {
        const long long e = base + 8ll * (i * kThreads + threadIdx.x);
        for (int j = 0; j < 8; ++j) {
          if (e + j >= T.n) break;
          const float v = value(T, e + j);
          sum[j] = fmaf(v, v, sum[j]);
        }
      }
    }
  }
  double total = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) total += sum[j];
  total = block_sum(total, s_sum);
  if (threadIdx.x == 0) __stcg(L.parts + L.part_begin + blockIdx.x, total);
}

__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ ClipLaunch L) {
  __shared__ double s_sum[kThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  double total = 0.0;
  for (int i = threadIdx.x; i < L.n_parts; i += kThreads) total += __ldcg(L.parts + i);
  const float norm = static_cast<float>(sqrt(block_sum(total, s_sum)));
  if (L.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *L.norm = norm;
  const float ratio = L.max_norm / (norm + L.eps);
  const float c = ratio >= 1.f ? 1.f : ratio;         // (a norm that is NaN stays one)
  if (L.in_place && c == 1.f) return;
  for (long long u = L.total_units - 1 - blockIdx.x; u >= 0; u -= gridDim.x) {
    const ClipTensor& T = tensor_of(L, u);
    const long long base = (u - T.unit_begin) * kClipUnit;
    if (base + kClipUnit <= T.n) {
      Raw r[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) load(T, base + 8ll * (i * kThreads + threadIdx.x), r[i]);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        float v[8];
        get(T, r[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= c;
        store(T, base + 8ll * (i * kThreads + threadIdx.x), v);
      }
    } else {
      for (int i = 0; i < kVecs; ++i) {
        const long long e = base + 8ll * (i * kThreads + threadIdx.x);
        for (int j = 0; j < 8; ++j) {
          if (e + j >= T.n) break;
          const float v = value(T, e + j) * c;
          if (T.out_bf16) static_cast<__nv_bfloat16*>(T.out)[e + j] = __float2bfloat16_rn(v);
          else static_cast<float*>(T.out)[e + j] = v;
        }
      }
    }
  }
}

cudaError_t launch_dependent(void (*kernel)(const ClipLaunch), int blocks, cudaStream_t s,
                             const ClipLaunch& l) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, l);
}

}  // namespace

int clip_blocks(const ClipLaunch& l, int sms) {
  return static_cast<int>(std::max<long long>(
      1, std::min<long long>({l.total_units, 4ll * sms, kClipBlocks})));
}

cudaError_t launch_grad_squares(const ClipLaunch& l, int blocks, cudaStream_t s) {
  return launch_dependent(grad_squares_kernel, blocks, s, l);
}

cudaError_t launch_clip(const ClipLaunch& l, int sms, cudaStream_t s) {
  return launch_dependent(clip_kernel, clip_blocks(l, sms), s, l);
}

}  // namespace muon
