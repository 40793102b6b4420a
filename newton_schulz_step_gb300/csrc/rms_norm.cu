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
// 16384 tokens of 2048 (bf16, with residual): forward 41.8 us (6.4 TB/s, 95 % of the copy's
// rate), gradients 49.2 (5.5 TB/s, the sum of the weight's parts among it); of 4096 in 8 bits
// 75.9 us (6.2 TB/s).  Blocks of 32 resident warps an SM forward (64 registers) gained 3 to 9 %
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

// ------------------------------------------------------------ rows whose squares leave the range
// A row whose mean square and eps together lie outside of [2^-38, 2^112) may be scaled by a
// power of two before its squares are summed: past 2^128 their sum would make every element 0, and
// below 2^-126 squares lose bits or vanish (where eps does not cover them).  The scale s brings the
// larger of the row's largest magnitude and eps^1/2 to [1, 4), so that nothing that counts leaves
// the range.  A row with an element that is not finite keeps s = 1.
// A team does its rows of that kind after the others, from memory, two or three times over; its loop
// pays a comparison: 16384 rows of 2048 take 41.8 us forward (41.6 without), 49.2 (48.8) backward,
// with 8 bits and no residual 26.7 (26.0), rows of 64 up to 4 % more.  (With the row scaled inside the
// loop, in registers, calls took up to a third longer.)  With a residual such a row's y is that of h
// as stored, one rounding more than in other rows: the sum may lie over what it was made of.
// All threads of a team go or none: it goes by the team's sum.
// The scale is taken outside of twice that range, by h as stored, which rounding has moved less: so
// it is by the row alone, and not by its neighbours, whether its y comes from the loop.  (The sum of
// 16384 squares is below 2^127 while their mean is below 2^113.)
constexpr float kLeastMean = 0x1p-38f, kMostMean = 0x1p112f;
static_assert(kRmsNormMaxDim <= 1 << 14, "sums of squares of rows in range");
__device__ __forceinline__ bool in_range(float mean) {
  return mean >= kLeastMean && mean < kMostMean;
}
__device__ __forceinline__ bool near_range(float mean) {
  return mean > 0.5f * kLeastMean && mean < 2.f * kMostMean;
}
// s for the row's largest magnitude as bits.
__device__ __forceinline__ float row_scale(uint32_t top, float eps) {
  if (top >= 0x7f800000u) return 1.f;
  const uint32_t e = max(top, __float_as_uint(sqrtf(eps))) >> 23;
  return __uint_as_float((254u - min(e, 253u)) << 23);
}
template <typename T>
__device__ __forceinline__ void load_row(const void* p, long long stride, int row, int c,
                                         float (&v)[8]) {
  Raw<T> r;
  r.load(static_cast<const T*>(p) + row * stride + 8 * c);
  r.get(v);
}
__device__ __forceinline__ void weight_times(const float* w, int c, float (&v)[8]) {
  if (w == nullptr) return;
  float m[8];
  load_row<float>(w, 0, 0, c, m);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= m[j];
}

// The thread's team, worked out anew with the thread's index behind the compiler's back: values kept
// for what follows the kernels' loops would spill some of the loops' own.
__device__ __forceinline__ Team new_team(const RmsNormLaunch& L, float* sums) {
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  Team team;
  team.threads = L.team;
  team.index = tid / L.team;
  team.at = tid - team.index * L.team;
  team.s = sums + team.index * (L.team >> 5) * 4;
  return team;
}

// The team's rows forward: of all of them (kSome) those that take the scale, or every row from `row`
// on (those that take none get the bits that the loop would give).
template <typename T, Mode kMode, bool kRes, bool kSome>
__device__ __forceinline__ void far_rows(const RmsNormLaunch& L, int row) {
  __shared__ float s_sums[kMaxTeam / 32 * 4];
  Team team = new_team(L, s_sums);
  const int vecs = L.dim >> 3, teams = blockDim.x / L.team, stride = gridDim.x * teams;
  if (kSome) row = blockIdx.x * teams + team.index;
  const void* const src = kRes ? L.sum : L.x;
  const long long src_stride = kRes ? L.sum_stride : L.x_stride;
  float h[8];
  auto top_of = [&] {
    uint32_t a = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(h[j]) & 0x7fffffffu);
    return a;
  };
#pragma unroll 1
  for (; row < L.tokens; row += stride) {
    float s = 1.f, r = 0.f;
    bool near = false;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {           // as it is; scaled
      uint32_t top = 0u;
      float ss = 0.f, unused = 0.f;
#pragma unroll 1
      for (int c = team.at; c < vecs; c += team.threads) {
        load_row<T>(src, src_stride, row, c, h);
        top = max(top, top_of());
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[j] * s, h[j] * s, ss);
      }
      team.sum2(ss, unused);
      const float mean = fmaf(ss, 1.f / static_cast<float>(L.dim), L.eps * s * s);
      r = rsqrtf(mean);
      if (pass == 0) {
        near = near_range(mean);
        if (near) break;
        s = row_scale(team.max1(top), L.eps);
      }
    }
    if (kSome && near) continue;
    float scale = 1.f;
    // 8 bits, a scale a row: its largest y first
#pragma unroll 1
    for (int pass = kMode == kEightBits && L.group == 0 ? 0 : 1; pass < 2; ++pass) {
      uint32_t top = 0u;
#pragma unroll 1
      for (int c = team.at; c - team.at < vecs; c += team.threads) {
        const bool on = c < vecs;                    // (all lanes of a warp, for the shuffles)
        if (on) {
          load_row<T>(src, src_stride, row, c, h);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] = h[j] * s * r;
          weight_times(L.w, c, h);
        }
        if constexpr (kMode == kForward) {
          if (on) Raw<T>::store(static_cast<T*>(L.y) + row * L.y_stride + 8 * c, h);
        } else {
          uint32_t a = on ? top_of() : 0u;
          top = max(top, a);
          if (pass == 0) continue;
          if (L.group != 0) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            scale = scale_of(a);
            if (on && (c & 15) == 0)
              L.scales[static_cast<size_t>(row) * L.groups + (c >> 4)] = scale;
          }
          const float inv = inverse(scale);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] *= inv;
          if (on)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(L.y) + row * L.y_stride + 8 * c) =
                e4m3_of(h);
        }
      }
      if (kMode == kEightBits && pass == 0) {
        scale = scale_of(team.max1(top));
        if (team.at == 0) L.scales[row] = scale;
      }
    }
  }
}

// The team's rows from `row` on, of the gradients; their terms of dw are added to those of the
// thread's vectors.
template <typename T>
__device__ __noinline__ void far_rows_backward(const RmsNormLaunch& L, int row, float* dw) {
  __shared__ float s_sums[kMaxTeam / 32 * 4];
  Team team = new_team(L, s_sums);
  const int vecs = L.dim >> 3, stride = gridDim.x * (blockDim.x / L.team);
  const float inv_dim = 1.f / static_cast<float>(L.dim);
#pragma unroll 1
  for (; row < L.tokens; row += stride) {
    float h[8], g[8], s = 1.f, r = 0.f, m = 0.f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {             // as it is; scaled
      uint32_t top = 0u;
      float ss = 0.f, gh = 0.f;
#pragma unroll 1
      for (int c = team.at; c < vecs; c += team.threads) {
        load_row<T>(L.x, L.x_stride, row, c, h);
        load_row<T>(L.dy, L.dy_stride, row, c, g);
        weight_times(L.w, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top = max(top, __float_as_uint(h[j]) & 0x7fffffffu);
          ss = fmaf(h[j] * s, h[j] * s, ss);
          // (h s is about 1: divided before it is added, the sum stays in the range of G's)
          gh = fmaf(pass == 0 ? g[j] : g[j] * inv_dim, h[j] * s, gh);
        }
      }
      team.sum2(ss, gh);
      const float mean = fmaf(ss, inv_dim, L.eps * s * s);
      r = rsqrtf(mean);
      m = -r * (pass == 0 ? gh * inv_dim : gh);
      if (pass == 0) {
        if (in_range(mean) && isfinite(gh)) break;     // a row after the one that led here
        s = row_scale(team.max1(top), L.eps);
      }
    }
    const float r_out = r * s;
#pragma unroll 1
    for (int i = 0, c = team.at; c < vecs; ++i, c += team.threads) {
      load_row<T>(L.x, L.x_stride, row, c, h);
      load_row<T>(L.dy, L.dy_stride, row, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = h[j] * s * r;
        dw[8 * i + j] = fmaf(g[j], h[j], dw[8 * i + j]);
      }
      weight_times(L.w, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = r_out * fmaf(h[j], m, g[j]);
      if (L.res != nullptr) {
        float e[8];
        load_row<T>(L.res, L.res_stride, row, c, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += e[j];
      }
      Raw<T>::store(static_cast<T*>(L.y) + row * L.y_stride + 8 * c, g);
    }
  }
}

// (Two blocks of 512, or four of 256, an SM: 64 registers.  Two bf16 vectors a thread with residual
// spill 4 bytes for it, and 16 with 8 bits.)
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
  // Rows out of range: whether there were any, where the call leaves what they are read from (the
  // sum with a residual, x for 8 bits); else the first one, from which on nothing is stored (out may
  // be x).
  constexpr bool kSome = kRes || kMode == kEightBits;
  bool any_far = false;
  int far = L.tokens;
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
    const float mean = fmaf(ss, inv_dim, L.eps);
    if constexpr (kSome) any_far |= !in_range(mean);
    else if (!in_range(mean)) far = min(far, row);
    const bool live = kSome || row < far;
    const float r = rsqrtf(mean);
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = team.at + i * L.team;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] *= r;
      if (c < vecs) w.times(i, c, h[i]);
      if constexpr (kMode == kForward) {
        if (live && c < vecs)
          Raw<T>::store(static_cast<T*>(L.y) + row * L.y_stride + 8 * c, h[i]);
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
  if constexpr (kSome) {
    if (any_far) far_rows<T, kMode, kRes, true>(L, 0);
  } else {
    if (far < L.tokens) far_rows<T, kMode, kRes, false>(L, far);
  }
}

// (Four vectors a thread spill, 56 bytes in bf16 and 248 in fp32, and have no row ahead: rows of 8192
// move at 4.7 TB/s, of 16384 at 3.2.)
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
    const float mean = fmaf(ss, inv_dim, L.eps);
    if (!in_range(mean) || !isfinite(gh)) break;         // (G h may leave the range without h^2)
    const float r = rsqrtf(mean);
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
  if (row < L.tokens) {
    float copy[kV * 8];
#pragma unroll
    for (int i = 0; i < kV * 8; ++i) copy[i] = dw[i / 8][i % 8];
    far_rows_backward<T>(L, row, copy);
#pragma unroll
    for (int i = 0; i < kV * 8; ++i) dw[i / 8][i % 8] = copy[i];
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
