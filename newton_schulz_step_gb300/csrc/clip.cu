// clip.cu -- the norm of all gradients of a model together, and the gradients clipped by it:
//
//   norm = (sum over all tensors and elements of g^2)^1/2
//   out  = g c,  c = min(1, max_norm / (norm + eps)), 1 where max_norm is infinite
//
// Two passes over the gradients, both bound by HBM: squares summed into one part a block,
// then the factor (every block adds the few hundred parts, in order) and the products.  The
// second pass walks the gradients backwards: it starts with what the first read last and L2
// still holds, and its own stores are marked to leave L2 first.  Gradients of up to about
// 100 MB are read from HBM once that way.  407 M bf16 gradients: 111 us (7.3 TB/s) and 232 (the
// reads and writes that reach HBM at 6.2 TB/s); 20 M in 47 tensors: 14.8 us together, of which
// the bytes at the copy's rate take 9.
//
// Squares are taken and added in fp32: a thread's sums are eight chains of at most 512 squares
// (past 2^128 the norm is infinite, which magnitudes below 2^58 do not reach; a magnitude below
// 2^-75 adds nothing), which are put into a total in one of two units after that many.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kClipUnit / 8 / kThreads;      // vectors of 8 a thread and unit

// 8 elements as stored.  kBf16: every gradient of the launch is bf16, so that half the
// registers hold them and all vectors of a unit travel at once; else half a unit does.
template <bool kBf16> struct Raw;
template <> struct Raw<true> {
  uint4 a;
};
template <> struct Raw<false> {
  uint4 a, b;                                        // b: fp32 only
};
template <bool kBf16> constexpr int kFlight = kBf16 ? kVecs : kVecs / 2;

__device__ __forceinline__ void load(const ClipTensor& T, long long e, Raw<true>& r) {
  r.a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(T.g) + e));
}
__device__ __forceinline__ void load(const ClipTensor& T, long long e, Raw<false>& r) {
  if (T.g_bf16) {
    r.a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(T.g) + e));
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(T.g) + e);
    r.a = __ldcg(p);
    r.b = __ldcg(p + 1);
  }
}
__device__ __forceinline__ void widen(const uint4& x, float (&v)[8]) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void get(const ClipTensor&, const Raw<true>& r, float (&v)[8]) {
  widen(r.a, v);
}
__device__ __forceinline__ void get(const ClipTensor& T, const Raw<false>& r, float (&v)[8]) {
  if (T.g_bf16) {
    widen(r.a, v);
    return;
  }
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
// Up to 8 elements from e on; those past the tensor are 0.
__device__ __forceinline__ void load_some(const ClipTensor& T, long long e, float (&v)[8]) {
  if (e + 8 <= T.n) {
    Raw<false> r;
    load(T, e, r);
    get(T, r, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.f;
    if (e + j < T.n)
      v[j] = T.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(T.g)[e + j])
                      : static_cast<const float*>(T.g)[e + j];
  }
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

// The launch's table of tensors in shared memory: a search among a kernel's arguments is a
// chain of misses of the constant cache, and this copy, before the wait for the kernel before,
// costs nothing.  (Read through a generic address: a different word a lane.)
__device__ __forceinline__ void load_table(const ClipLaunch& L, ClipTensor* table) {
  static_assert(sizeof(ClipTensor) % 8 == 0, "whole words");
  const unsigned long long* from = reinterpret_cast<const unsigned long long*>(&L.t[0]);
  asm("" : "+l"(from));
  unsigned long long* to = reinterpret_cast<unsigned long long*>(table);
  const int words = L.n_tensors * static_cast<int>(sizeof(ClipTensor) / 8);
  for (int i = threadIdx.x; i < words; i += kThreads) to[i] = from[i];
}
// Tensor of unit u: the last one that begins at or before it.
__device__ __forceinline__ const ClipTensor& tensor_of(const ClipTensor* table, int n, long long u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid].unit_begin <= u) lo = mid;
    else hi = mid - 1;
  }
  return table[lo];
}

// Sums of squares pass fp32's range before their root does.  They are held in fp32 in units of 1,
// or of 2^40 once a thread's exceeds 2^96: fp64 runs at a sixtieth of fp32's rate here, and adding
// the threads' sums in it took longer than reading the gradients (40 MB: 15 us, 9 without).
constexpr float kLarge = 0x1p96f, kUnit = 0x1p-40f;
// Units of 8 squares a chain between which a thread's chains go into its totals: gradients of up to
// 64 x 608 x 16384 elements (637 M) need no such step.
constexpr int kFoldUnits = 64;
static_assert(kFoldUnits * kVecs == 512, "squares of a chain");
// Sum over the block, the same for every thread and run.
__device__ __forceinline__ float block_sum(float x, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) x += s[k];
  return x;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) grad_squares_kernel(const __grid_constant__ ClipLaunch L) {
  __shared__ float s_sum[kThreads / 32];
  __shared__ ClipTensor s_table[kMaxClipTensors];
  ptx::griddep_launch_dependents();
  load_table(L, s_table);
  __syncthreads();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
  float plain = 0.f, scaled = 0.f;                   // totals of earlier chains, in units of 1 and 2^40
  int units = 0;
  for (long long u = blockIdx.x; u < L.total_units; u += gridDim.x) {
    if (units++ == kFoldUnits) {
      units = 1;
      bool large = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) large |= sum[j] > kLarge;
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t += large ? sum[j] * kUnit : sum[j];
        sum[j] = 0.f;
      }
      (large ? scaled : plain) += t;
    }
    const ClipTensor& T = tensor_of(s_table, L.n_tensors, u);
    const long long base = (u - T.unit_begin) * kClipUnit;
    if (base + kClipUnit <= T.n) {
#pragma unroll 1
      for (int p = 0; p < kVecs; p += kFlight<kBf16>) {
        Raw<kBf16> r[kFlight<kBf16>];
#pragma unroll
        for (int i = 0; i < kFlight<kBf16>; ++i)
          load(T, base + 8ll * ((p + i) * kThreads + threadIdx.x), r[i]);
#pragma unroll
        for (int i = 0; i < kFlight<kBf16>; ++i) {
          float v[8];
          get(T, r[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[j] = fmaf(v[j], v[j], sum[j]);
        }
      }
    } else {
      // a tensor's last unit: whole vectors, then up to 7 elements
#pragma unroll 2
      for (int i = 0; i < kVecs; ++i) {
        const long long e = base + 8ll * (i * kThreads + threadIdx.x);
        if (e >= T.n) break;
        float v[8];
        load_some(T, e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(v[j], v[j], sum[j]);
      }
    }
  }
  bool over = plain > kLarge || scaled != 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) over |= sum[j] > kLarge;
  const int large = __syncthreads_or(over);
  float total = large ? fmaf(plain, kUnit, scaled) : plain;
#pragma unroll
  for (int j = 0; j < 8; ++j) total += large ? sum[j] * kUnit : sum[j];
  total = block_sum(total, s_sum);
  if (threadIdx.x == 0) {
    __stcg(L.parts + L.part_begin + blockIdx.x, make_float2(total, __int_as_float(large)));
  }
}

// (64 registers, for four blocks an SM; the bf16 form spills 32 bytes for it.)
template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) clip_kernel(const __grid_constant__ ClipLaunch L) {
  __shared__ float s_sum[kThreads / 32];
  __shared__ ClipTensor s_table[kMaxClipTensors];
  ptx::griddep_launch_dependents();
  load_table(L, s_table);
  __syncthreads();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  // a block's first whole unit travels while the parts are added
  long long u = L.total_units - 1 - blockIdx.x;
  Raw<kBf16> r[kFlight<kBf16>];
  auto fetch = [&](const ClipTensor& T, long long base) {
#pragma unroll
    for (int i = 0; i < kFlight<kBf16>; ++i)
      load(T, base + 8ll * (i * kThreads + threadIdx.x), r[i]);
  };
  bool fetched = false;
  if (u >= 0) {
    const ClipTensor& T = tensor_of(s_table, L.n_tensors, u);
    const long long base = (u - T.unit_begin) * kClipUnit;
    fetched = base + kClipUnit <= T.n;
    if (fetched) fetch(T, base);
  }
  float plain = 0.f, scaled = 0.f;                   // parts in units of 1, and of 2^40
  bool over = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < L.n_parts; i += kThreads) {
    const float2 p = __ldcg(L.parts + i);
    const bool large = __float_as_int(p.y) != 0;
    over |= large;
    plain += large ? 0.f : p.x;
    scaled += large ? p.x : 0.f;
  }
  const int large = __syncthreads_or(over);
  const float total = block_sum(large ? fmaf(plain, kUnit, scaled) : plain, s_sum);
  const float norm = large ? sqrtf(total) * 0x1p20f : sqrtf(total);
  if (L.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *L.norm = norm;
  // (infinity over a norm that is not finite would be NaN; a norm that is NaN stays one)
  const float ratio = isinf(L.max_norm) ? 1.f : L.max_norm / (norm + L.eps);
  const float c = ratio >= 1.f ? 1.f : ratio;
  if (L.in_place && c == 1.f) return;
  for (; u >= 0; u -= gridDim.x) {
    const ClipTensor& T = tensor_of(s_table, L.n_tensors, u);
    const long long base = (u - T.unit_begin) * kClipUnit;
    if (c == 1.f && T.out == T.g) {                   // in place: it stays as it is
      fetched = false;
      continue;
    }
    if (base + kClipUnit <= T.n) {
#pragma unroll 1
      for (int p = 0; p < kVecs; p += kFlight<kBf16>) {
        const long long at = base + 8ll * p * kThreads;
        if (!fetched) fetch(T, at);
        fetched = false;
#pragma unroll
        for (int i = 0; i < kFlight<kBf16>; ++i) {
          float v[8];
          get(T, r[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= c;
          store(T, at + 8ll * (i * kThreads + threadIdx.x), v);
        }
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < kVecs; ++i) {
        const long long e = base + 8ll * (i * kThreads + threadIdx.x);
        if (e >= T.n) break;
        float v[8];
        load_some(T, e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= c;
        if (e + 8 <= T.n) {
          store(T, e, v);
        } else {
          for (int j = 0; j < 8 && e + j < T.n; ++j) {
            if (T.out_bf16) static_cast<__nv_bfloat16*>(T.out)[e + j] = __float2bfloat16_rn(v[j]);
            else static_cast<float*>(T.out)[e + j] = v[j];
          }
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

static bool all_bf16(const ClipLaunch& l) {
  for (int i = 0; i < l.n_tensors; ++i)
    if (!l.t[i].g_bf16) return false;
  return true;
}

cudaError_t launch_grad_squares(const ClipLaunch& l, int blocks, cudaStream_t s) {
  return launch_dependent(all_bf16(l) ? grad_squares_kernel<true> : grad_squares_kernel<false>,
                          blocks, s, l);
}

cudaError_t launch_clip(const ClipLaunch& l, int sms, cudaStream_t s) {
  return launch_dependent(all_bf16(l) ? clip_kernel<true> : clip_kernel<false>,
                          clip_blocks(l, sms), s, l);
}

}  // namespace muon
