// rms_norm.cu -- the residual's addition and the RMS norm of the sum, with an output in the
// inputs' type or in 8 bits with scales, and the gradients.
//
//   h = x + residual,   y = h r w,   r = (mean h^2 + eps)^-1/2
//   8 bits: y = s q a group of columns (or a row), q in e4m3, s the least power of two that
//           brings the group's largest |y| to 448 or less
//   dx = r (G - h r mean(G h r)) + dresidual,  G = dy w;   dw = sum over tokens of dy h r
//
// All of it is bound by HBM: each element is read once and written once.  A row is held in
// registers by a team of 32 to 512 threads, vectors of 8 elements a thread: one pass over
// the data, one sum over the team (the gradients' two sums travel together).  Teams of a
// block work on rows of their own; the rows' loads are issued a row ahead, so that they
// travel while the row before is summed.  A power of two as the scale makes the division
// exact: the only rounding is e4m3's own, and the values that q stands for are exact in bf16.
//
// 16384 tokens of 2048 (bf16, with residual): forward 41.4 us (6.5 TB/s, 96 % of the copy's
// rate), gradients 49.0 (5.5 TB/s, the sum of the weight's parts among it); of 4096 in 8 bits
// 75.5 us (6.2 TB/s).  Blocks of 32 resident warps an SM forward (64 registers) gained 3 to 9 %
// over 24; the gradients keep 16, their columns' sums of the weight take the registers.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;        // of a block; 512 where a row's team has as many
constexpr int kMaxTeam = 512;

// 8 elements of a row as stored.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// A team of `threads` (a power of two, 32..512) and its scratch: sums of two rows' worth, so
// that one barrier a sum is enough (a slot is written again two sums later).
struct Team {
  int threads, index, at;              // size, team of the block, thread of the team
  float* s;                            // [2 slots][warps of the team][2]
  int slot = 0;
  __device__ __forceinline__ void sync() const {
    if (threads == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
  }
  __device__ __forceinline__ void sum2(float& a, float& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (threads == 32) return;
    const int warps = threads >> 5, w = at >> 5;
    float* const p = s + slot * 2 * warps;
    if ((at & 31) == 0) {
      p[2 * w] = a;
      p[2 * w + 1] = b;
    }
    sync();
    a = b = 0.f;
    for (int i = 0; i < warps; ++i) {
      a += p[2 * i];
      b += p[2 * i + 1];
    }
    slot ^= 1;
  }
  __device__ __forceinline__ uint32_t max1(uint32_t a) {
    a = __reduce_max_sync(0xffffffffu, a);
    if (threads == 32) return a;
    const int warps = threads >> 5;
    uint32_t* const p = reinterpret_cast<uint32_t*>(s + slot * 2 * warps);
    if ((at & 31) == 0) p[at >> 5] = a;
    sync();
    for (int i = 0; i < warps; ++i) a = max(a, p[i]);
    slot ^= 1;
    return a;
  }
};

// 2^e for the group's largest |y| (its bits): the least power of two with |y| <= 448 2^e.
// 448 = 1.75 2^8.  0 gives 1, what is not finite NaN: the whole group then reads as NaN.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax == 0u) return 1.f;
  if (amax >= 0x7f800000u) return __int_as_float(0x7fffffff);
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __int_as_float(max(e, 1) << 23);
}
// q = y / s for s = 2^e, -126 <= e <= 120: the inverse is a power of two as well.
__device__ __forceinline__ float inverse(float s) {
  return s == s ? __int_as_float((254 << 23) - __float_as_int(s)) : s;
}
__device__ __forceinline__ uint2 e4m3_of(const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    h[i] = r;
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// Weights of a thread's vectors: in registers while these are few.
template <int kV>
struct Weights {
  static constexpr bool kHeld = kV <= 2;
  float v[kHeld ? kV : 1][8];
  const float* w;
  __device__ __forceinline__ void init(const float* weight, int at, int threads, int vecs) {
    w = weight;
    if constexpr (kHeld) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = at + i * threads;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 1.f;
        if (w != nullptr && c < vecs) fetch(c, v[i]);
      }
    }
  }
  __device__ __forceinline__ void fetch(int c, float (&o)[8]) const {
    Raw<float> x;
    x.a = __ldg(reinterpret_cast<const float4*>(w + 8 * c));
    x.b = __ldg(reinterpret_cast<const float4*>(w + 8 * c + 4));
    x.get(o);
  }
  __device__ __forceinline__ void times(int i, int c, float (&o)[8]) const {
    if (w == nullptr) return;
    float m[8];
    if constexpr (kHeld) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = v[i][j];
    } else {
      fetch(c, m);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] *= m[j];
  }
};

enum Mode { kForward, kEightBits };

template <typename T, Mode kMode, int kV, bool kRes>
__global__ void __launch_bounds__(kMaxTeam, sizeof(T) == 2 ? 2 : 1) rms_norm_kernel(const __grid_constant__ RmsNormLaunch L) {
  constexpr bool kAhead = kV <= 2;     // a row ahead in registers
  __shared__ float s_sums[kMaxTeam / 32 * 4];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  Team team;
  team.threads = L.team;
  team.index = threadIdx.x / L.team;
  team.at = threadIdx.x - team.index * L.team;
  team.s = s_sums + team.index * (L.team >> 5) * 4;
  const int vecs = L.dim >> 3;
  const float inv_dim = 1.f / static_cast<float>(L.dim);
  Weights<kV> w;
  w.init(L.w, team.at, L.team, vecs);
  const int teams = blockDim.x / L.team, stride = gridDim.x * teams;
  const T* const x = static_cast<const T*>(L.x);
  const T* const res = static_cast<const T*>(L.res);   // (kRes)

  Raw<T> rx[kV], rr[kRes ? kV : 1];
  auto load = [&](int row) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
      rx[i].clear();
      if constexpr (kRes) rr[i].clear();
      if (row < L.tokens && c < vecs) {
        rx[i].load(x + row * L.x_stride + 8 * c);
        if constexpr (kRes) rr[i].load(res + row * L.res_stride + 8 * c);
      }
    }
  };
  int row = blockIdx.x * teams + team.index;
  if (kAhead) load(row);
  for (; row < L.tokens; row += stride) {
    if (!kAhead) load(row);
    float h[kV][8];
    float ss = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
      rx[i].get(h[i]);
      if constexpr (kRes) {
        float r[8];
        rr[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        if (c < vecs) Raw<T>::store(static_cast<T*>(L.sum) + row * L.sum_stride + 8 * c, h[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    if (kAhead) load(row + stride);
    team.sum2(ss, unused);
    const float r = rsqrtf(fmaf(ss, inv_dim, L.eps));
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] *= r;
      if (c < vecs) w.times(i, c, h[i]);
      if constexpr (kMode == kForward) {
        if (c < vecs) Raw<T>::store(static_cast<T*>(L.y) + row * L.y_stride + 8 * c, h[i]);
      } else {
        // the largest magnitude as bits: NaN above Inf above what is finite
        uint32_t a = 0u;
        if (c < vecs) {
#pragma unroll
          for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(h[i][j]) & 0x7fffffffu);
        }
        if (L.group == 0) {
          top = max(top, a);
        } else {
          // 128 columns are 16 lanes
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
          const float s = scale_of(a), inv = inverse(s);
          if (c < vecs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= inv;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(L.y) + row * L.y_stride + 8 * c) =
                e4m3_of(h[i]);
            if ((c & 15) == 0) L.scales[static_cast<size_t>(row) * L.groups + (c >> 4)] = s;
          }
        }
      }
    }
    if constexpr (kMode == kEightBits) {
      if (L.group == 0) {
        const float s = scale_of(team.max1(top)), inv = inverse(s);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int c = team.at + i * L.team;
          if (c < vecs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= inv;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(L.y) + row * L.y_stride + 8 * c) =
                e4m3_of(h[i]);
          }
        }
        if (team.at == 0) L.scales[row] = s;
      }
    }
  }
}

// dx and a block's part of dw.  The team of a row keeps its columns' sums of dy h r; the
// teams' sums are added in order, and rms_norm_weight_kernel adds the blocks'.
template <typename T, int kV>
__global__ void __launch_bounds__(kMaxTeam)
    rms_norm_backward_kernel(const __grid_constant__ RmsNormLaunch L) {
  constexpr bool kAhead = kV * sizeof(T) <= 4;   // (two fp32 vectors ahead do not fit)
  extern __shared__ float s_dw[];      // [teams][dim], where there is a weight
  __shared__ float s_sums[kMaxTeam / 32 * 4];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  Team team;
  team.threads = L.team;
  team.index = threadIdx.x / L.team;
  team.at = threadIdx.x - team.index * L.team;
  team.s = s_sums + team.index * (L.team >> 5) * 4;
  const int vecs = L.dim >> 3;
  const float inv_dim = 1.f / static_cast<float>(L.dim);
  Weights<kV> w;
  w.init(L.w, team.at, L.team, vecs);
  const int teams = blockDim.x / L.team, stride = gridDim.x * teams;
  const T* const x = static_cast<const T*>(L.x);       // h as stored
  const T* const dy = static_cast<const T*>(L.dy);
  const T* const res = static_cast<const T*>(L.res);   // dresidual
  float dw[kV][8];
#pragma unroll
  for (int i = 0; i < kV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;

  Raw<T> rx[kV], rg[kV], rr[kV];
  auto load = [&](int row) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
      rx[i].clear();
      rg[i].clear();
      rr[i].clear();
      if (row < L.tokens && c < vecs) {
        rx[i].load(x + row * L.x_stride + 8 * c);
        rg[i].load(dy + row * L.dy_stride + 8 * c);
        if (res != nullptr) rr[i].load(res + row * L.res_stride + 8 * c);
      }
    }
  };
  int row = blockIdx.x * teams + team.index;
  if (kAhead) load(row);
  for (; row < L.tokens; row += stride) {
    if (!kAhead) load(row);
    float h[kV][8], g[kV][8];
    Raw<T> rres[kV];
    float ss = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      rx[i].get(h[i]);
      rg[i].get(g[i]);
      rres[i] = rr[i];
      float gw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) gw[j] = g[i][j];
      const int c = team.at + i * L.team;
      if (c < vecs) w.times(i, c, gw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(h[i][j], h[i][j], ss);
        gh = fmaf(gw[j], h[i][j], gh);
      }
    }
    if (kAhead) load(row + stride);
    team.sum2(ss, gh);
    const float r = rsqrtf(fmaf(ss, inv_dim, L.eps));
    const float m = -r * (gh * inv_dim);                 // (r^2 may overflow, h r does not)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
      if (c >= vecs) continue;
      float o[8], e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] *= r;
        dw[i][j] = fmaf(g[i][j], h[i][j], dw[i][j]);
        o[j] = g[i][j];
      }
      w.times(i, c, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r * fmaf(h[i][j], m, o[j]);
      if (res != nullptr) {
        rres[i].get(e);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += e[j];
      }
      Raw<T>::store(static_cast<T*>(L.y) + row * L.y_stride + 8 * c, o);
    }
  }
  if (L.parts == nullptr) return;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = team.at + i * L.team;
    if (c < vecs) Raw<float>::store(s_dw + team.index * L.dim + 8 * c, dw[i]);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < L.dim; d += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < teams; ++k) s += s_dw[k * L.dim + d];
    __stcg(L.parts + static_cast<size_t>(blockIdx.x) * L.dim + d, s);
  }
}

// dw = sum of the blocks' parts, in a fixed order: 32 columns a block, 32 warps that take every
// 32nd part each (all of a warp's loads in flight at once).
__global__ void __launch_bounds__(1024)
    rms_norm_weight_kernel(const float* parts, int blocks, int dim, float* dw,
                           const unsigned int* status) {
  __shared__ float s_sum[32][33];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(status)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  constexpr int kEach = (kRmsNormMaxBlocks + 31) / 32;
  float v[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = warp + 32 * i;
    v[i] = b < blocks && d < dim ? __ldcg(parts + static_cast<size_t>(b) * dim + d) : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) s += v[i];
  s_sum[warp][lane] = s;
  __syncthreads();
  s = s_sum[lane][warp];                     // column `warp`, one lane a warp's sum
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + warp < dim) dw[blockIdx.x * 32 + warp] = s;
}

template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, int blocks, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Threads of a row's team: two vectors a thread, while that makes 32 to `most` of them.
int team_of(int dim, int most) {
  int t = 32;
  while (t < most && 2 * t < dim / 8) t *= 2;
  return t;
}
// Forward, four vectors a thread and more blocks on an SM are better than a row ahead (4096 rows
// of 8192: 43 us with teams of 256, 51 with 512); backward it is the other way (88 and 58).
int forward_team(int dim) { return team_of(dim, dim / 8 <= 4 * kThreads ? kThreads : kMaxTeam); }
int backward_team(int dim) { return team_of(dim, kMaxTeam); }
int threads_of(int team) { return std::max(team, kThreads); }

template <typename T, Mode kMode, bool kRes>
cudaError_t forward_as(const RmsNormLaunch& l, int sms, cudaStream_t s) {
  const int threads = threads_of(l.team), per = threads / l.team;
  const int each = (l.dim / 8 + l.team - 1) / l.team;
  const int blocks = std::min((l.tokens + per - 1) / per, 8 * sms);
  auto go = [&](auto kernel) { return launch_dependent(kernel, blocks, threads, 0, s, l); };
  if (each <= 1) return go(rms_norm_kernel<T, kMode, 1, kRes>);
  if (each <= 2) return go(rms_norm_kernel<T, kMode, 2, kRes>);
  return go(rms_norm_kernel<T, kMode, 4, kRes>);
}
template <typename T, Mode kMode>
cudaError_t forward(const RmsNormLaunch& l, int sms, cudaStream_t s) {
  return l.res != nullptr ? forward_as<T, kMode, true>(l, sms, s)
                          : forward_as<T, kMode, false>(l, sms, s);
}

template <typename T>
cudaError_t backward(const RmsNormLaunch& l, int blocks, cudaStream_t s) {
  const int threads = threads_of(l.team), each = (l.dim / 8 + l.team - 1) / l.team;
  const int smem = l.parts != nullptr ? threads / l.team * l.dim * 4 : 0;
  auto go = [&](auto kernel) -> cudaError_t {
    if (smem > 48 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, blocks, threads, smem, s, l);
  };
  if (each <= 1) return go(rms_norm_backward_kernel<T, 1>);
  if (each <= 2) return go(rms_norm_backward_kernel<T, 2>);
  return go(rms_norm_backward_kernel<T, 4>);
}

}  // namespace

cudaError_t launch_rms_norm(RmsNormLaunch l, bool bf16, bool eight_bits, int sms, cudaStream_t s) {
  l.team = forward_team(l.dim);
  if (bf16)
    return eight_bits ? forward<__nv_bfloat16, kEightBits>(l, sms, s)
                      : forward<__nv_bfloat16, kForward>(l, sms, s);
  return eight_bits ? forward<float, kEightBits>(l, sms, s) : forward<float, kForward>(l, sms, s);
}

int rms_norm_blocks(int tokens, int dim) {
  const int team = backward_team(dim), per = threads_of(team) / team;
  return std::min((tokens + per - 1) / per, kRmsNormMaxBlocks);
}

cudaError_t launch_rms_norm_backward(RmsNormLaunch l, bool bf16, cudaStream_t s) {
  l.team = backward_team(l.dim);
  const int blocks = rms_norm_blocks(l.tokens, l.dim);
  return bf16 ? backward<__nv_bfloat16>(l, blocks, s) : backward<float>(l, blocks, s);
}

cudaError_t launch_rms_norm_weight(const RmsNormLaunch& l, float* dw, cudaStream_t s) {
  return launch_dependent(rms_norm_weight_kernel, (l.dim + 31) / 32, 1024, 0, s,
                          static_cast<const float*>(l.parts), rms_norm_blocks(l.tokens, l.dim),
                          l.dim, dw, l.status);
}

}  // namespace muon
