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
// written once.  A row (one head of one token) is held by G = head_dim / 8 (rounded
// up to a power of two) lanes, 8 elements each; a warp takes kIter x (32 / G)
// consecutive rows, first all of the queries', then of the keys', and issues their
// loads before it uses the first.  With the half layout a lane's 8 elements are 4 + 4,
// rot / 2 apart, so that both members of a pair are in one thread: the rotation needs
// no exchange, and only the sum of squares (backward: also the mean of G h) crosses
// lanes.  The table rows are read for every head, from L1 after a token's first.
// Waiting rows stay in their storage type, which keeps a thread within 64 registers
// and 32 warps on an SM: that many loads in flight cover the memory's latency.
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// rows of a lane at a time: 4 x 16 bytes in flight (backward: 2 x 2 x 16)
template <typename T, bool kBackward> constexpr int kIter = (kBackward ? 4 : 8) / sizeof(T);
template <bool kBackward> constexpr int kResident = kBackward ? 3 : 4;   // blocks on an SM
constexpr int kPartGroups = 32;      // first level of the weight gradients' sum
constexpr int kGroupMax = kRopeMaxBlocks / kPartGroups;   // blocks per group
static_assert(kGroupMax * kPartGroups == kRopeMaxBlocks, "groups cover the blocks");

struct Vec8 { float v[8]; };

// 8 elements of a row as stored: two groups of 4, or 8 contiguous ones.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <bool kWhole> __device__ __forceinline__ void load(const float* p, int ea, int eb) {
    a = *reinterpret_cast<const float4*>(p + ea);
    b = *reinterpret_cast<const float4*>(p + eb);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  template <bool kWhole>
  static __device__ __forceinline__ void store(float* p, int ea, int eb, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p + ea) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + eb) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void clear() { a = b = make_uint2(0, 0); }
  template <bool kWhole>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int ea, int eb) {
    if constexpr (kWhole) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + ea);
      a = make_uint2(x.x, x.y);
      b = make_uint2(x.z, x.w);
    } else {
      a = *reinterpret_cast<const uint2*>(p + ea);
      b = *reinterpret_cast<const uint2*>(p + eb);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const unsigned int w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  template <bool kWhole>
  static __device__ __forceinline__ void store(__nv_bfloat16* p, int ea, int eb,
                                               const float (&v)[8]) {
    unsigned int w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned int*>(&x);
    }
    if constexpr (kWhole) {
      *reinterpret_cast<uint4*>(p + ea) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(p + ea) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(p + eb) = make_uint2(w[2], w[3]);
    }
  }
};

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
__global__ void __launch_bounds__(kThreads, kResident<kBackward>)
    norm_rope_kernel(const __grid_constant__ NormRopeLaunch L) {
  constexpr int kN = kIter<T, kBackward>;
  __shared__ float s_dw[kBackward ? kWarps * 2 * kRopeMaxDim : 1];
  __shared__ int s_last;
  if (kBackward && ptx::status_set(L.status)) return;   // the same word for every thread: set
                                                        // words stay set until the host clears
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = L.dim >> 3;                       // 8-element units of a row
  const int g = units <= 1 ? 1 : 1 << (32 - __clz(units - 1));   // lanes of a row
  const int u = lane & (g - 1);                       // this lane's unit
  const int sub = lane / g, per = 32 / g;             // row within the warp, rows at a time
  const bool on = u < units;
  const bool rotated = u < (L.rot >> 3);
  const int ea = !kInterleaved && rotated ? 4 * u : 8 * u;            // first 4 elements
  const int eb = !kInterleaved && rotated ? (L.rot >> 1) + 4 * u : 8 * u + 4;
  const float inv_dim = 1.f / static_cast<float>(L.dim);
  const int width = 2 * L.dim;

  if constexpr (kBackward) {
    if (L.dw[0] != nullptr || L.dw[1] != nullptr)
      for (int d = lane; d < width; d += 32) s_dw[warp * width + d] = 0.f;
    __syncwarp();
  }

  int unit = blockIdx.x * kWarps + warp, passed = 0;  // work units; those of the kinds before
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int heads = L.heads[s];
    if (heads == 0) continue;
    const int rows = L.tokens * heads;
    const int count = (rows + kN * per - 1) / (kN * per);
    const int dt = per / heads, dh = per - dt * heads;   // from a row to the one `per` on
    float w[8], dw[kBackward ? 8 : 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if constexpr (kBackward) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] = 0.f;
    }
    if (on && L.w[s] != nullptr) {
      Raw<float> x;
      x.template load<false>(L.w[s], ea, eb);
      x.get(w);
    }
    for (; unit - passed < count; unit += gridDim.x * kWarps) {
      const int row0 = (unit - passed) * (kN * per) + sub;
      const int t0 = row0 / heads, h0 = row0 - t0 * heads;
      Raw<T> x[kN], dy[kBackward ? kN : 1];
#pragma unroll
      for (int i = 0, t = t0, h = h0; i < kN; ++i) {
        const bool live = on && row0 + i * per < rows;
        x[i].clear();
        if (live && (!kBackward || L.norm))
          x[i].template load<kInterleaved>(
              static_cast<const T*>(L.x[s].p) + t * L.x[s].ts + h * L.x[s].hs, ea, eb);
        if constexpr (kBackward) {
          dy[i].clear();
          if (live)
            dy[i].template load<kInterleaved>(
                static_cast<const T*>(L.dy[s].p) + t * L.dy[s].ts + h * L.dy[s].hs, ea, eb);
        }
        t += dt;
        h += dh;
        if (h >= heads) {
          h -= heads;
          ++t;
        }
      }
#pragma unroll
      for (int i = 0, t = t0, h = h0; i < kN; ++i) {
        const bool live = on && row0 + i * per < rows;
        float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
        float poison = 1.f;                           // NaN for a position outside the tables
        if (L.rot > 0 && live) {
          const int pos = L.pos != nullptr ? __ldg(L.pos + t) : t;
          if (pos < 0 || pos >= L.table_len) {
            poison = __int_as_float(0x7fffffff);
          } else if (rotated) {
            const size_t at = static_cast<size_t>(pos) * (L.rot >> 1) + 4 * u;
            const float4 a = __ldg(reinterpret_cast<const float4*>(L.cos + at));
            const float4 b = __ldg(reinterpret_cast<const float4*>(L.sin + at));
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
            sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
          }
        }
        float xv[8], o[8], r = 1.f;
        x[i].get(xv);
        if (L.norm) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(xv[j], xv[j], ss);
          r = rsqrtf(fmaf(head_sum(ss, g), inv_dim, L.eps));
          if (!live) r = 0.f;                         // (rsqrt(0) of a row that is not there)
        }
        if constexpr (!kBackward) {
          r *= poison;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = xv[j] * r * w[j];
          if (rotated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = o[first<kInterleaved>(j)], b = o[second<kInterleaved>(j)];
              o[first<kInterleaved>(j)] = a * c[j] - b * sn[j];
              o[second<kInterleaved>(j)] = b * c[j] + a * sn[j];
            }
          }
        } else {
          dy[i].get(o);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= poison;
          if (rotated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = o[first<kInterleaved>(j)], b = o[second<kInterleaved>(j)];
              o[first<kInterleaved>(j)] = a * c[j] + b * sn[j];
              o[second<kInterleaved>(j)] = b * c[j] - a * sn[j];
            }
          }
          if (L.norm) {
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              xv[j] *= r;
              dw[j] = fmaf(o[j], xv[j], dw[j]);
              o[j] *= w[j];
              dot = fmaf(o[j], xv[j], dot);
            }
            dot = head_sum(dot, g) * inv_dim;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = r * (o[j] - xv[j] * dot);
          }
        }
        if (live)
          Raw<T>::template store<kInterleaved>(
              static_cast<T*>(L.y[s].p) + t * L.y[s].ts + h * L.y[s].hs, ea, eb, o);
        t += dt;
        h += dh;
        if (h >= heads) {
          h -= heads;
          ++t;
        }
      }
    }
    passed += count;
    if constexpr (kBackward) {
      if (L.dw[s] != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = dw[j];
          for (int o = g; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (sub == 0 && on) s_dw[warp * width + s * L.dim + (j < 4 ? ea + j : eb + j - 4)] = v;
        }
      }
    }
  }

  if constexpr (kBackward) {
    if (L.dw[0] == nullptr && L.dw[1] == nullptr) return;
    // Weight gradients, in a fixed order: lanes, warps, then blocks in two levels of
    // at most 19 and 32 rows (each level's loads in flight together; one block
    // summing 608 rows alone would take 608 / (loads in flight) memory latencies).
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
  const long long chunk = kIter<T, kBackward> * (32 / g);
  long long total = 0;
  for (int h : l.heads) total += (1ll * l.tokens * h + chunk - 1) / chunk;
  const long long want = (total + kWarps - 1) / kWarps;
  const int cap = min(kRopeMaxBlocks, kResident<kBackward> * sms);
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
