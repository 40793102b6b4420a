// norm_rope.cu -- RMS norm and rotary position embedding of every query and key
// head in one pass, and their gradients.
//
// Forward, per token and head: n = x r w with r = (mean x^2 + eps)^-1/2, then the
// pairs of the first `rot` elements are rotated by the token's angle.  Backward:
// with g = the output's gradient rotated back, h = x r and G = g w,
//   dw = sum g h (tokens, heads),   dx = r (G - h mean(G h)).
// r is recomputed from x, which the backward pass reads in any case.
//
// Both are bound by HBM: every element is read once (backward: x and dy) and
// written once.  A warp takes one token and up to kIter x (32 / G) of its heads,
// so that the token's table rows are read once and stay in registers; a head's
// G = head_dim / 8 (rounded up to a power of two) lanes hold 8 elements each.
// With the half layout those 8 are 4 + 4 elements, rot / 2 apart, so that both
// members of a pair are in one thread: the rotation needs no exchange, and only
// the sum of squares (backward: also the mean of G h) crosses lanes.  All loads of
// a warp's heads are issued before the first is used.
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kIter = 4;             // heads a lane works on at a time
constexpr int kPartGroups = 32;      // first level of the weight gradients' sum
constexpr int kGroupMax = kRopeMaxBlocks / kPartGroups;   // blocks per group
static_assert(kGroupMax * kPartGroups == kRopeMaxBlocks, "groups cover the blocks");

struct Vec8 { float v[8]; };

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const unsigned int*>(&a),
                                            *reinterpret_cast<const unsigned int*>(&b));
}

// index in Vec8 of the first and second member of pair j
template <bool kInterleaved> __device__ __forceinline__ constexpr int first(int j) {
  return kInterleaved ? 2 * j : j;
}
template <bool kInterleaved> __device__ __forceinline__ constexpr int second(int j) {
  return kInterleaved ? 2 * j + 1 : j + 4;
}

// Sum over the `g` (power of two) lanes of a head.
__device__ __forceinline__ float head_sum(float x, int g) {
  for (int o = g >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sums rows [r0, r1) of parts ([row][width]) into column d, all loads in flight.
template <int kMax>
__device__ __forceinline__ float sum_rows(const float* parts, int r0, int r1, int width, int d) {
  float v[kMax];
#pragma unroll
  for (int i = 0; i < kMax; ++i)
    v[i] = r0 + i < r1 ? __ldcg(parts + static_cast<size_t>(r0 + i) * width + d) : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMax; ++i) s += v[i];
  return s;
}

template <typename T, bool kBackward, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeLaunch L) {
  __shared__ float s_dw[kBackward ? kWarps * 2 * kRopeMaxDim : 1];
  __shared__ int s_last;
  if (kBackward && ptx::status_set(L.status)) return;   // the same word for every thread: set
                                                        // words stay set until the host clears
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = L.dim >> 3;                       // 8-element units of a head
  const int g = units <= 1 ? 1 : 1 << (32 - __clz(units - 1));   // lanes of a head
  const int u = lane & (g - 1);                       // this lane's unit
  const int sub = lane / g, per = 32 / g;             // head within the warp, heads at a time
  const bool on = u < units;
  const bool rotated = u < (L.rot >> 3);
  const int ea = !kInterleaved && rotated ? 4 * u : 8 * u;            // first 4 elements
  const int eb = !kInterleaved && rotated ? (L.rot >> 1) + 4 * u : 8 * u + 4;
  const int heads = L.heads[0] + L.heads[1];
  const int chunk_heads = kIter * per;
  const int chunks = (heads + chunk_heads - 1) / chunk_heads;
  const int total = L.tokens * chunks;
  const float inv_dim = 1.f / static_cast<float>(L.dim);

  Vec8 w[2], dw[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[s].v[j] = 1.f;
      dw[s].v[j] = 0.f;
    }
    if (on && L.w[s] != nullptr) {
      load4(L.w[s] + ea, w[s].v);
      load4(L.w[s] + eb, w[s].v + 4);
    }
  }

  for (int unit = blockIdx.x * kWarps + warp; unit < total; unit += gridDim.x * kWarps) {
    const int t = unit / chunks;
    const int h0 = (unit - t * chunks) * chunk_heads + sub;
    Vec8 x[kIter], dy[kBackward ? kIter : 1];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int hh = h0 + i * per;
      const int s = hh >= L.heads[0];
      const int h = s ? hh - L.heads[0] : hh;
      const bool live = on && hh < heads;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].v[j] = 0.f;
      if (live && (!kBackward || L.norm)) {
        const T* p = static_cast<const T*>(L.x[s].p) + t * L.x[s].ts + h * L.x[s].hs;
        load4(p + ea, x[i].v);
        load4(p + eb, x[i].v + 4);
      }
      if constexpr (kBackward) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[i].v[j] = 0.f;
        if (live) {
          const T* p = static_cast<const T*>(L.dy[s].p) + t * L.dy[s].ts + h * L.dy[s].hs;
          load4(p + ea, dy[i].v);
          load4(p + eb, dy[i].v + 4);
        }
      }
    }
    float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    float poison = 1.f;                               // NaN for a position outside the tables
    if (L.rot > 0) {
      const int pos = L.pos != nullptr ? L.pos[t] : t;
      if (pos < 0 || pos >= L.table_len) {
        poison = __int_as_float(0x7fffffff);
      } else if (rotated) {
        const size_t at = static_cast<size_t>(pos) * (L.rot >> 1) + 4 * u;
        load4(L.cos + at, c);
        load4(L.sin + at, sn);
      }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int hh = h0 + i * per;
      const int s = hh >= L.heads[0];
      const int h = s ? hh - L.heads[0] : hh;
      const bool live = on && hh < heads;
      float r = 1.f;
      if (L.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[i].v[j], x[i].v[j], ss);
        r = rsqrtf(fmaf(head_sum(ss, g), inv_dim, L.eps));
      }
      Vec8 o;
      if constexpr (!kBackward) {
        r *= poison;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = x[i].v[j] * r * (s ? w[1].v[j] : w[0].v[j]);
        if (rotated) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = o.v[first<kInterleaved>(j)], b = o.v[second<kInterleaved>(j)];
            o.v[first<kInterleaved>(j)] = a * c[j] - b * sn[j];
            o.v[second<kInterleaved>(j)] = b * c[j] + a * sn[j];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = dy[i].v[j] * poison;
        if (rotated) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = o.v[first<kInterleaved>(j)], b = o.v[second<kInterleaved>(j)];
            o.v[first<kInterleaved>(j)] = a * c[j] + b * sn[j];
            o.v[second<kInterleaved>(j)] = b * c[j] - a * sn[j];
          }
        }
        if (L.norm) {
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = x[i].v[j] * r;
            const float gh = live ? o.v[j] * xh : 0.f;   // (poison is NaN on idle lanes too)
            if (s) dw[1].v[j] += gh;
            else dw[0].v[j] += gh;
            o.v[j] *= s ? w[1].v[j] : w[0].v[j];
            if (live) dot = fmaf(o.v[j], xh, dot);
          }
          dot = head_sum(dot, g) * inv_dim;
#pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] = r * (o.v[j] - x[i].v[j] * r * dot);
        }
      }
      if (live) {
        T* p = static_cast<T*>(L.y[s].p) + t * L.y[s].ts + h * L.y[s].hs;
        store4(p + ea, o.v);
        store4(p + eb, o.v + 4);
      }
    }
  }

  if constexpr (kBackward) {
    if (L.dw[0] == nullptr && L.dw[1] == nullptr) return;
    // Weight gradients, in a fixed order: lanes, warps, then blocks in two levels of
    // at most 19 and 32 rows (each level's loads in flight together; one block
    // summing 608 rows alone would take 608 / (loads in flight) memory latencies).
    const int width = 2 * L.dim;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = dw[s].v[j];
        for (int o = g; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0 && on) s_dw[warp * width + s * L.dim + (j < 4 ? ea + j : eb + j - 4)] = v;
      }
    __syncthreads();
    for (int d = threadIdx.x; d < width; d += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += s_dw[k * width + d];
      __stcg(L.parts + static_cast<size_t>(blockIdx.x) * width + d, v);
    }
    const int nb = static_cast<int>(gridDim.x);
    const int group = blockIdx.x / kGroupMax, groups = (nb + kGroupMax - 1) / kGroupMax;
    const int b0 = group * kGroupMax, b1 = min(nb, b0 + kGroupMax);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = atomicInc(L.ticket + 1 + group, b1 - b0 - 1) == static_cast<unsigned>(b1 - b0 - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float* sums = L.parts + static_cast<size_t>(kRopeMaxBlocks) * width;
    for (int d = threadIdx.x; d < width; d += kThreads)
      __stcg(sums + static_cast<size_t>(group) * width + d,
             sum_rows<kGroupMax>(L.parts, b0, b1, width, d));
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = atomicInc(L.ticket, groups - 1) == static_cast<unsigned>(groups - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int d = threadIdx.x; d < width; d += kThreads) {
      const int s = d >= L.dim;
      if (L.dw[s] != nullptr)
        L.dw[s][d - s * L.dim] = sum_rows<kPartGroups>(sums, 0, groups, width, d);
    }
  }
}

template <typename T, bool kBackward>
cudaError_t launch(const NormRopeLaunch& l, int sms, cudaStream_t s) {
  int units = l.dim >> 3, g = 1;
  while (g < units) g <<= 1;
  const int heads = l.heads[0] + l.heads[1];
  const int chunk = kIter * (32 / g);
  const long long total = 1ll * l.tokens * ((heads + chunk - 1) / chunk);
  const long long want = (total + kWarps - 1) / kWarps;
  const int cap = kBackward ? min(kRopeMaxBlocks, 4 * sms) : 8 * sms;
  const int blocks = static_cast<int>(want < cap ? want : cap);
  if (l.interleaved) norm_rope_kernel<T, kBackward, true><<<blocks, kThreads, 0, s>>>(l);
  else norm_rope_kernel<T, kBackward, false><<<blocks, kThreads, 0, s>>>(l);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& l, bool backward, int sms, cudaStream_t s) {
  if (l.bf16)
    return backward ? launch<__nv_bfloat16, true>(l, sms, s)
                    : launch<__nv_bfloat16, false>(l, sms, s);
  return backward ? launch<float, true>(l, sms, s) : launch<float, false>(l, sms, s);
}

}  // namespace muon
