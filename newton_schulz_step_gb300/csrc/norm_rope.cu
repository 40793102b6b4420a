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
// lanes.  Waiting rows stay in their storage type, the arithmetic is on fp32 pairs.
// What held earlier forms back was the chain position -> table row -> first row: without
// it the forward of 32768 tokens, 32 + 8 heads of 128, took 111 us instead of 146 (the
// bytes alone: 101).  So a position is read a step ahead, and the table row with the rows
// it belongs to: 138 us; with the lanes of a row known at compile time and no division
// a step 121 us (5.7 TB/s with the tables and positions, 84 % of the copy rate).
// Backward of 16384 tokens, 16 + 16 heads of 128: 86 us (4.8 TB/s, 70 %).  What holds the
// rest is that a warp loads, then computes, with too few others beside it: issue slots 60 %
// with 24 warps an SM forward (about 150 instructions for 8 elements), 51 % with 16 backward
// (250), waits for loads the first of the stalls.
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Rows of a lane at a time, and blocks on an SM: 4 x 16 bytes in flight in 24 warps, or
// (backward) 4 x 2 x 16 in 16 warps.  (Backward with half the rows in 24 warps: 90 us
// instead of 86 at the size above; forward with twice the rows in 16 warps: 125 instead of
// 121.)
template <typename T> constexpr int kIter = 8 / sizeof(T);
template <bool kBackward> constexpr int kResident = kBackward ? 2 : 3;
constexpr int kPartGroups = 32;      // first level of the weight gradients' sum
constexpr int kGroupMax = kRopeMaxBlocks / kPartGroups;   // blocks per group
static_assert(kGroupMax * kPartGroups == kRopeMaxBlocks, "groups cover the blocks");

using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

__device__ __forceinline__ uint64_t pair_of(uint32_t w) {   // two bf16
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_of(uint64_t v) {
  const float2 f = unpair(v);
  const __nv_bfloat162 x = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
  const float2 f = unpair(v);
  return pair(f.y, f.x);
}
__device__ __forceinline__ float sum_of(uint64_t v) {
  const float2 f = unpair(v);
  return f.x + f.y;
}

// 8 elements of a row as stored, in two groups of 4 (kWhole: 8 contiguous ones); in
// fp32 they are four pairs.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <bool kWhole> __device__ __forceinline__ void load(const float* p, int ea, int eb) {
    a = *reinterpret_cast<const float4*>(p + ea);
    b = *reinterpret_cast<const float4*>(p + eb);
  }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    v[0] = pair(a.x, a.y); v[1] = pair(a.z, a.w);
    v[2] = pair(b.x, b.y); v[3] = pair(b.z, b.w);
  }
  template <bool kWhole>
  static __device__ __forceinline__ void store(float* p, int ea, int eb, const uint64_t (&v)[4]) {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = unpair(v[i]);
    *reinterpret_cast<float4*>(p + ea) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    *reinterpret_cast<float4*>(p + eb) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
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
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    v[0] = pair_of(a.x); v[1] = pair_of(a.y);
    v[2] = pair_of(b.x); v[3] = pair_of(b.y);
  }
  template <bool kWhole>
  static __device__ __forceinline__ void store(__nv_bfloat16* p, int ea, int eb,
                                               const uint64_t (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_of(v[i]);
    if constexpr (kWhole) {
      *reinterpret_cast<uint4*>(p + ea) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(p + ea) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(p + eb) = make_uint2(w[2], w[3]);
    }
  }
};

// The rotation of a lane's four (a, b) by angles with cosines c and sines s.  Half
// layout: pairs 0, 1 hold the a, pairs 2, 3 the b.  Interleaved: a pair holds (a, b), and
// the cosines and sines come doubled, the sines of a with their sign changed.
template <bool kInterleaved> struct Angles;
template <> struct Angles<false> {
  uint64_t c[2], s[2], ms[2];
  __device__ __forceinline__ void set(const float4& x, const float4& y) {
    c[0] = pair(x.x, x.y); c[1] = pair(x.z, x.w);
    s[0] = pair(y.x, y.y); s[1] = pair(y.z, y.w);
    ms[0] = pair(-y.x, -y.y); ms[1] = pair(-y.z, -y.w);
  }
  __device__ __forceinline__ void turn(uint64_t (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = v[i], b = v[2 + i];
      v[i] = fma2(b, ms[i], mul2(a, c[i]));
      v[2 + i] = fma2(a, s[i], mul2(b, c[i]));
    }
  }
  __device__ __forceinline__ void turn_back(uint64_t (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = v[i], b = v[2 + i];
      v[i] = fma2(b, s[i], mul2(a, c[i]));
      v[2 + i] = fma2(a, ms[i], mul2(b, c[i]));
    }
  }
};
template <> struct Angles<true> {
  uint64_t c[4], s[4];
  __device__ __forceinline__ void set(const float4& x, const float4& y) {
    c[0] = pair(x.x, x.x); c[1] = pair(x.y, x.y); c[2] = pair(x.z, x.z); c[3] = pair(x.w, x.w);
    s[0] = pair(-y.x, y.x); s[1] = pair(-y.y, y.y);
    s[2] = pair(-y.z, y.z); s[3] = pair(-y.w, y.w);
  }
  __device__ __forceinline__ void turn(uint64_t (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(swapped(v[i]), s[i], mul2(v[i], c[i]));
  }
  __device__ __forceinline__ void turn_back(uint64_t (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(swapped(v[i]), swapped(s[i]), mul2(v[i], c[i]));
  }
};

// Sum over the `g` (power of two) lanes of a row; kLanes: g, or 0 where it is not known
// at compile time.
template <int kLanes>
__device__ __forceinline__ float head_sum(float x, int g) {
#pragma unroll
  for (int o = kLanes ? kLanes / 2 : 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    if (kLanes || o < g) x += y;
  }
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

template <typename T, bool kBackward, bool kInterleaved, int kLanes>
__global__ void __launch_bounds__(kThreads, kResident<kBackward>)
    norm_rope_kernel(const __grid_constant__ NormRopeLaunch L) {
  constexpr int kN = kIter<T>;
  __shared__ float s_dw[kBackward ? kWarps * 2 * kRopeMaxDim : 1];
  __shared__ int s_last;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();                 // the kernel before, which may still have been running
  if (kBackward && ptx::status_set(L.status)) return;   // the same word for every thread: set
                                                        // words stay set until the host clears
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = L.dim >> 3;                       // 8-element units of a row
  const int g = kLanes ? kLanes : units <= 1 ? 1 : 1 << (32 - __clz(units - 1));   // of a row
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
#pragma unroll
  for (int s = 0; s < 2; ++s) {                       // (unrolled: the strides stay constants)
    const int heads = L.heads[s];
    if (heads == 0) continue;
    const int rows = L.tokens * heads;
    const int count = (rows + kN * per - 1) / (kN * per);
    const int dt = per / heads, dh = per - dt * heads;   // from a row to the one `per` on
    uint64_t w[4], dw[kBackward ? 4 : 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pair(1.f, 1.f);
    if constexpr (kBackward) {
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[j] = 0;
    }
    if (on && L.w[s] != nullptr) {
      Raw<float> x;
      x.template load<false>(L.w[s], ea, eb);
      x.get(w);
    }
    // from a row to the one `per` on: a step, and a correction where the token changes
    const long long xs = L.x[s].ts * dt + L.x[s].hs * dh, xw = L.x[s].ts - L.x[s].hs * heads;
    const long long ys = L.y[s].ts * dt + L.y[s].hs * dh, yw = L.y[s].ts - L.y[s].hs * heads;
    const long long gs = L.dy[s].ts * dt + L.dy[s].hs * dh, gw = L.dy[s].ts - L.dy[s].hs * heads;
    // position of token t, -1 outside the tables
    auto position = [&](int t) {
      const int pos = L.pos != nullptr ? __ldg(L.pos + t) : t;
      return pos >= 0 && pos < L.table_len ? pos : -1;
    };
    const int stride = gridDim.x * kWarps;
    int row0 = (unit - passed) * (kN * per) + sub, t0 = row0 / heads, h0 = row0 - t0 * heads;
    const int row_step = stride * (kN * per), t_step = row_step / heads;
    const int h_step = row_step - t_step * heads;      // (a division a step cost 25 instructions)
    int pos0 = L.rot > 0 && t0 < L.tokens ? position(t0) : 0;
    for (; unit - passed < count; unit += stride) {
      Raw<T> x[kN], dy[kBackward ? kN : 1];
      {
        const T* px = static_cast<const T*>(L.x[s].p) + t0 * L.x[s].ts + h0 * L.x[s].hs;
        const T* pg = kBackward
            ? static_cast<const T*>(L.dy[s].p) + t0 * L.dy[s].ts + h0 * L.dy[s].hs : nullptr;
        int h = h0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const bool live = on && row0 + i * per < rows;
          x[i].clear();
          if (live && (!kBackward || L.norm)) x[i].template load<kInterleaved>(px, ea, eb);
          if constexpr (kBackward) {
            dy[i].clear();
            if (live) dy[i].template load<kInterleaved>(pg, ea, eb);
          }
          px += xs;
          if constexpr (kBackward) pg += gs;
          h += dh;
          if (h >= heads) {
            h -= heads;
            px += xw;
            if constexpr (kBackward) pg += gw;
          }
        }
      }
      // the first row's angles travel with the rows: its position was read a step ahead
      float4 cosines = make_float4(1.f, 1.f, 1.f, 1.f), sines = make_float4(0.f, 0.f, 0.f, 0.f);
      auto table_row = [&](int pos) {
        const size_t at = static_cast<size_t>(pos) * (L.rot >> 1) + 4 * u;
        cosines = __ldg(reinterpret_cast<const float4*>(L.cos + at));
        sines = __ldg(reinterpret_cast<const float4*>(L.sin + at));
      };
      if (rotated && pos0 >= 0) table_row(pos0);
      int next_t0 = t0 + t_step, next_h0 = h0 + h_step;
      if (next_h0 >= heads) {
        next_h0 -= heads;
        ++next_t0;
      }
      int next_pos0 = 0;
      if (L.rot > 0 && unit - passed + stride < count && next_t0 < L.tokens)
        next_pos0 = position(next_t0);
      T* py = static_cast<T*>(L.y[s].p) + t0 * L.y[s].ts + h0 * L.y[s].hs;
      Angles<kInterleaved> angles;
      if (rotated) angles.set(cosines, sines);
      float poison = pos0 < 0 ? __int_as_float(0x7fffffff) : 1.f;   // outside the tables: NaN
      int t = t0, h = h0, have = t0;                  // `have`: the token of `angles`
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const bool live = on && row0 + i * per < rows;
        if (L.rot > 0 && live && t != have) {
          have = t;
          const int pos = position(t);
          poison = pos < 0 ? __int_as_float(0x7fffffff) : 1.f;
          if (rotated && pos >= 0) {
            table_row(pos);
            angles.set(cosines, sines);
          }
        }
        uint64_t v[4], o[4];
        float r = 1.f;
        x[i].get(v);
        if (L.norm) {
          const uint64_t ss = fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0]))));
          r = rsqrtf(fmaf(head_sum<kLanes>(sum_of(ss), g), inv_dim, L.eps));
          if (!live) r = 0.f;                         // (rsqrt(0) of a row that is not there)
        }
        if constexpr (!kBackward) {
          const uint64_t r2 = pair(r * poison, r * poison);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = mul2(mul2(v[j], r2), w[j]);
          if (rotated) angles.turn(o);
        } else {
          const uint64_t r2 = pair(r, r);
          dy[i].get(o);
          // (lanes past the head, and rows that are not there, keep their zeros: they enter the
          // sums of rows whose position is good)
          if (__builtin_expect(live && poison != 1.f, 0)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = pair(poison, poison);
          }
          if (rotated) angles.turn_back(o);
          if (L.norm) {
            uint64_t dot = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = mul2(v[j], r2);
              dw[j] = fma2(o[j], v[j], dw[j]);       // (rows that are not there: 0)
              o[j] = mul2(o[j], w[j]);
              dot = fma2(o[j], v[j], dot);
            }
            const float m = -head_sum<kLanes>(sum_of(dot), g) * inv_dim;
            const uint64_t m2 = pair(m, m);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = mul2(r2, fma2(v[j], m2, o[j]));
          }
        }
        if (live) Raw<T>::template store<kInterleaved>(py, ea, eb, o);
        py += ys;
        t += dt;
        h += dh;
        if (h >= heads) {
          h -= heads;
          ++t;
          py += yw;
        }
      }
      row0 += row_step;
      t0 = next_t0;
      h0 = next_h0;
      pos0 = next_pos0;
    }
    passed += count;
    if constexpr (kBackward) {
      if (L.dw[s] != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = j & 1 ? unpair(dw[j >> 1]).y : unpair(dw[j >> 1]).x;
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
  const long long chunk = kIter<T> * (32 / g);
  long long total = 0;
  for (int h : l.heads) total += (1ll * l.tokens * h + chunk - 1) / chunk;
  const long long want = (total + kWarps - 1) / kWarps;
  const int cap = min(kRopeMaxBlocks, kResident<kBackward> * sms);
  const int blocks = static_cast<int>(want < cap ? want : cap);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto with_lanes = [&](auto lanes) {
    constexpr int k = decltype(lanes)::value;
    return l.interleaved ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, kBackward, true, k>, l)
                         : cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, kBackward, false, k>, l);
  };
  return g == 8    ? with_lanes(std::integral_constant<int, 8>())
         : g == 16 ? with_lanes(std::integral_constant<int, 16>())
                   : with_lanes(std::integral_constant<int, 0>());
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& l, bool backward, int sms, cudaStream_t s) {
  if (l.bf16)
    return backward ? launch<__nv_bfloat16, true>(l, sms, s)
                    : launch<__nv_bfloat16, false>(l, sms, s);
  return backward ? launch<float, true>(l, sms, s) : launch<float, false>(l, sms, s);
}

}  // namespace muon
