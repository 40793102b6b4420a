// attention.cuh -- what the attention kernels share: the sequence that a token
// belongs to, shared-memory tiles, bounded waits, and one row of each result
// computed by a warp from its definition.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace attn {

using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBlock = 128;            // rows of a tile (keys or queries)
constexpr uint32_t kSlab = 16384;      // 128 rows x 64 bf16, 128-byte swizzle

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

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

// Tokens that belong to a sequence: those past them are padding.
__device__ __forceinline__ int tokens_in_use(const AttentionLaunch& L) {
  return L.cu == nullptr ? L.T : min(max(__ldg(L.cu + L.n_seqs), 0), L.T);
}

// The tile (every thread of the block calls this) whose work is the `want`-th largest: blocks
// start in the order of their index, and a long tile that starts last ends last.
// work(i): the blocks that tile i walks.
// It costs every block its searches and two barriers, 1 us and more with many tiles, and a
// wave the key blocks that neighbouring tiles share.  So it pays where documents of different
// lengths take few waves, and a wave holds several tiles (the heads of a tile are blocks that
// follow each other).  Time with it over time without, three packs of random lengths each:
//   forward   4096 tokens, 12/12 heads of 64 (1.3 waves)     0.97  0.92  1.05
//             8192 tokens, 8/4 heads of 64 (1.7)             0.85  0.80  0.98
//             8192 tokens, 12/12 heads of 64 (2.5)           0.98  1.01  1.04
//               (8 documents of 5 to 2400 tokens             0.94)
//             16384 tokens, 8/4 heads of 64 (3.4)            0.96  0.95  0.96
//             32768 tokens, 12/12 heads of 64 (10)           1.04  1.05  1.05
//             4096 tokens, 24/8 heads of 64 (2.5)            1.08  1.05  1.09
//   dq and dk, dv in a row, dk, dv ranked
//             4096 tokens, 24/8 heads of 64 (1.7 waves)      0.91  0.96  0.98
//             16384 tokens, 16/4 heads of 128 (3.4)          0.90  0.92  0.97
//             32768 tokens, 16/4 heads of 128 (6.7)          1.02  1.01  0.99
//             4096 tokens, 12/12 heads of 64 (2.5)           1.05  1.03  1.05
//               (a key head with one query head has short walks: not ranked there)
// dq, with a block for each query head, has many waves: 1.03 to 1.2, and it is not ranked.
constexpr int kRankedTiles = 256;        // the scratch of the ranking
inline bool rank_tiles(int n_seqs, int tiles, int heads, int sms) {
  const long long blocks = 1ll * tiles * heads;
  return n_seqs > 1 && tiles <= kRankedTiles && blocks > sms && blocks <= 4ll * sms &&
         8 * heads <= sms;
}
template <typename F>
__device__ __forceinline__ int ranked_tile(int tiles, int want, int* scratch, F&& work) {
  for (int i = threadIdx.x; i < tiles; i += blockDim.x) scratch[i] = work(i);
  __syncthreads();
  for (int i = threadIdx.x; i < tiles; i += blockDim.x) {
    const int w = scratch[i];
    int rank = 0;
    for (int k = 0; k < tiles; ++k) rank += scratch[k] > w || (scratch[k] == w && k < i);
    if (rank == want) scratch[kRankedTiles] = i;
  }
  ptx::fence_proxy_async_smem();         // copies will land where the scratch is
  __syncthreads();
  return __shfl_sync(0xffffffffu, scratch[kRankedTiles], 0);
}

// Launch that may begin before the kernel in front of it in the stream has ended: its
// blocks set up their barriers, then wait for that kernel (begin_after_prior) before they
// touch global memory or take TMEM, which that kernel may still need.  The three kernels
// of a training pass follow each other without the gap of a launch.
template <typename K>
cudaError_t launch_behind(K kernel, int blocks, int threads, uint32_t smem,
                          const AttentionMaps& m, const AttentionLaunch& l, cudaStream_t s,
                          int cluster = 1) {
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, m, l);
}
__device__ __forceinline__ void begin_after_prior() {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
}

// ---- bounded waits ------------------------------------------------------
// Every wait of a CTA goes through its abort flag and the workspace's status word:
// a wait that gives up sets both, which ends the waits of the CTA's other roles.
// The code of the issuing roles is kept short (waiting is a call there, loops stay
// loops): all roles share the instruction caches, and with everything unrolled every
// step of the issuing warp was measured to wait 300 cycles for its instructions.
static __device__ __noinline__ bool wait_call(uint64_t* bar, uint32_t parity,
                                              const volatile int* bad, unsigned int* status) {
  return ptx::mbar_wait(bar, parity, bad, status);
}

struct Guard {
  volatile int* bad;
  unsigned int* status;
  unsigned int role;                     // DeviceError bit of the waiting role
  __device__ __forceinline__ void fail() const {
    if (!*bad) atomicOr(status, kErrTimeoutAttention | role);
    *bad = 1;
  }
  // One issuing thread's wait; records a failure.
  __device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity) const {
    if (ptx::mbar_try_wait(bar, parity) || wait_call(bar, parity, bad, status)) return true;
    fail();
    return false;
  }
  // An issuing warp's wait (the lanes agree on the result).
  __device__ __forceinline__ bool issue_wait(uint64_t* bar, uint32_t parity) const {
    for (int i = 0; i < 8; ++i)          // (a try itself waits a while)
      if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, wait_call(bar, parity, bad, status))) return true;
    fail();
    return false;
  }
  // A compute warp's wait (a call would cost it the registers it holds).
  __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const {
    const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, bad, status));
    if (!ok) fail();
    return ok;
  }
};
// What a role still has in flight when it gives up is waited for, within this limit.
constexpr uint64_t kDrainNs = 100ull * 1000ull * 1000ull;

// The dynamic shared memory starts on the 1024 bytes that the swizzled tiles need (it
// follows the system's own 1 KB); a kernel that found it elsewhere would do nothing and
// report a failed wait.
__device__ __forceinline__ bool tiles_aligned(const uint8_t* sm) {
  return (ptx::smem_u32(sm) & 1023u) == 0;
}

// ---- tiles --------------------------------------------------------------
// A tile is 128 rows of one head in DP / 64 slabs of 64 columns, 128-byte swizzle:
// as a matrix operand it can be read along the head (K-major: 16 columns a step) or
// along its rows (MN-major: 16 rows a step).
template <int DP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int head, int row,
                                          uint64_t* bar) {
  ptx::mbar_arrive_expect_tx(bar, DP / 64 * kSlab);
#pragma unroll
  for (int s = 0; s < DP / 64; ++s) ptx::tma_load_3d(dst + s * kSlab, map, 64 * s, head, row, bar);
}
// Address of a tile for descriptors: the offset in the block's own shared memory.  (In a
// cluster, a shared-memory address also holds the block's rank, in bits that would reach
// into the descriptor's other fields.)
__device__ __forceinline__ uint32_t tile_address(const uint8_t* tile) {
  return ptx::smem_u32(tile) & 0x3FFFFu;
}
// Operand descriptors (ptx::smem_desc_sw128) with the tile's address added last, so that
// the steps of a product differ by a constant.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int step) {   // 16 columns from 16 step
  return ptx::smem_desc_sw128(0, 16, 1024) +
         ((tile + (step >> 2) * kSlab + (step & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int step) {  // 16 rows from 16 step
  return ptx::smem_desc_sw128(0, kSlab, 1024) + ((tile + step * 2048) >> 4);
}
// Position in a ring of `kN` slots.
template <int kN> struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kN) {
      slot = 0;
      parity ^= 1u;
    }
  }
};
// Products, issued by one elected lane of a warp in step.  A CTA holds all 512 TMEM
// columns, so their addresses start at 0.
// D = A B^T over the head: both tiles K-major
template <int DP>
__device__ __forceinline__ void mma_heads(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t kId = ptx::idesc_bf16(128, 128, false);
#pragma unroll 1
  for (uint32_t s = 0; s < DP / 64; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ptx::mma_bf16(d, desc_k(a + s * kSlab, i), desc_k(b + s * kSlab, i), kId, s > 0 || i > 0);
}
// The same with A in TMEM (bf16 pairs, DP / 2 columns): a product from shared memory alone
// reads 8 KB of it for 64 cycles of a 128 x 128 x 16 step, all that it delivers.
template <int DP>
__device__ __forceinline__ void mma_heads_ts(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t kId = ptx::idesc_bf16(128, 128, false);
#pragma unroll 1
  for (uint32_t s = 0; s < DP / 64; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ptx::mma_bf16_ts(d, a + 32 * s + 8 * i, desc_k(b + s * kSlab, i), kId, s > 0 || i > 0);
}
// D (+)= A[tmem] B over the first kRows rows of B.  A: bf16 pairs, kRun columns (of 32
// bits) from `a`, the next from a + 2 kRun, and so on
template <int DP, int kRows, int kRun>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  constexpr uint32_t kId = ptx::idesc_bf16(128, DP, true);
#pragma unroll 1
  for (uint32_t s = 0; s < kRows / 64; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ptx::mma_bf16_ts(d, a + 64 * s + 8 * i + 8 * i / kRun * kRun, desc_mn(b + s * 8192, i), kId,
                       accumulate || s > 0 || i > 0);
}
// byte offset of 8 elements (row, column 8 c) of a tile
__device__ __forceinline__ uint32_t tile_off(int row, int c) {
  return static_cast<uint32_t>(c >> 3) * kSlab + static_cast<uint32_t>(row) * 128u +
         ((static_cast<uint32_t>(c & 7) ^ static_cast<uint32_t>(row & 7)) << 4);
}
// Zeroes row `row` of a tile.  Tokens that no row of a block's tile sees (padding, and the
// sequences before or behind) may hold anything, and zero weights do not stop Inf or NaN in
// a product.  (fence_proxy_async_smem before the product reads it.)
template <int DP>
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
  for (int c = 0; c < DP / 8; ++c)
    *reinterpret_cast<uint4*>(tile + tile_off(row, c)) = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// 32 fp32 values as bf16 into columns 8 c .. 8 c + 31 of a row
__device__ __forceinline__ void store_row32(uint8_t* tile, int row, int c, const float (&f)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(tile + tile_off(row, c + q)) =
        make_uint4(pack2(f[8 * q], f[8 * q + 1]), pack2(f[8 * q + 2], f[8 * q + 3]),
                   pack2(f[8 * q + 4], f[8 * q + 5]), pack2(f[8 * q + 6], f[8 * q + 7]));
}

// Columns outside lo..hi become `value`: one mask a row, then a bit an element.  (With two
// compares an element the tile where one document ends and the next begins, which hides keys
// in every block it walks, held up the others: 8192 packed tokens, 16/4 heads of 128, dk/dv
// in 231 us instead of 190.)
__device__ __forceinline__ void hide(uint32_t (&s)[32], int lo, int hi, uint32_t value) {
  const uint32_t visible = (lo > 31 ? 0u : ~0u << max(lo, 0)) &
                           (hi < 0 ? 0u : ~0u >> (31 - min(hi, 31)));
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!(visible >> j & 1u)) s[j] = value;
}

// ---- rows by definition -------------------------------------------------
// A matrix product over a tile multiplies invisible pairs by a weight of zero, and zero
// times Inf or NaN is NaN.  Operand rows that no row of the tile sees are cleared; what is
// left to leak are tokens of the tile itself.  dk and dv know the queries that hold such
// values by their log-sum-exp and delta, and clear these too.  out and dq do not know the
// keys: a result row that is not finite is looked into by one warp.  It stays as it is where
// its own sequence says so (a visible weight is not finite, and with it the whole row, or a
// visible operand in the same column); otherwise it is computed again from its visible pairs
// alone.  Nothing of this runs on finite data.
// The looking keeps a diverged run from stalling: one row by definition takes 150 cycles a
// key, and a NaN in a document's first key reaches all its rows.  (2048 tokens, 8/4 heads of
// 64, every such row walked: 29 ms forward instead of 0.05.  What is walked now are a tile's
// rows before a bad token: 4 ms.)
// A lane holds the elements 2 lane, 2 lane + 1 of each 64-element half of a head.
struct Row { float v[4]; };
struct Packed { unsigned int w[2]; };    // the same in bf16

__device__ __forceinline__ Packed load_packed(const __nv_bfloat16* p, int dim) {
  const int lane = threadIdx.x & 31;
  Packed r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 64 * h + 2 * lane;
    r.w[h] = d < dim ? *reinterpret_cast<const unsigned int*>(p + d) : 0u;
  }
  return r;
}
__device__ __forceinline__ Row unpack(const Packed& x) {
  Row r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r.v[2 * h] = __uint_as_float(x.w[h] << 16);
    r.v[2 * h + 1] = __uint_as_float(x.w[h] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Row load_row(const __nv_bfloat16* p, int dim) {
  return unpack(load_packed(p, dim));
}

// Sums over the warp.
template <int kN> __device__ __forceinline__ void warp_sums(float (&s)[kN]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
}
__device__ __forceinline__ float dot_part(const Row& a, const Row& b) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(a.v[j], b.v[j], s);
  return s;
}
// acc += f x
__device__ __forceinline__ void axpy(Row& acc, float f, const Row& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc.v[j] = fmaf(f, x.v[j], acc.v[j]);
}

// Elements of this lane that are not finite, a bit each.
__device__ __forceinline__ unsigned int not_finite(const Packed& x) {
  unsigned int bad = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if ((x.w[h] & 0x7f80u) == 0x7f80u) bad |= 1u << 2 * h;
    if ((x.w[h] & 0x7f800000u) == 0x7f800000u) bad |= 2u << 2 * h;
  }
  return bad;
}
// Columns in which one of the rows a..b-1 of a head is not finite.
static __device__ __noinline__ unsigned int bad_columns(const Heads<const __nv_bfloat16>& x, int head,
                                                        int a, int b, int dim) {
  constexpr int kN = 16;                 // rows in flight
  unsigned int bad = 0;
  for (int t = a; t < b; t += kN) {
    Packed w[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) w[n] = load_packed(x.row(min(t + n, b - 1), head), dim);
#pragma unroll
    for (int n = 0; n < kN; ++n) bad |= not_finite(w[n]);
  }
  return bad;
}

// A row as bf16 in row `row` of a shared-memory tile.
__device__ __forceinline__ uint32_t* row_slot(uint8_t* tile, int row, int half) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<uint32_t*>(tile + tile_off(row, 8 * half + (lane >> 2)) +
                                     4 * (lane & 3));
}
__device__ __forceinline__ void put_row(uint8_t* tile, int row, const Row& r, int slabs) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (h < slabs) *row_slot(tile, row, h) = pack2(r.v[2 * h], r.v[2 * h + 1]);
}
__device__ __forceinline__ unsigned int bad_elements(uint8_t* tile, int row, int slabs) {
  Packed x = {{0u, 0u}};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (h < slabs) x.w[h] = *row_slot(tile, row, h);
  return not_finite(x);
}

// Output row i of query head h over the keys begin..i.
static __device__ __noinline__ Row out_row(const AttentionLaunch& L, int h, int i, int begin) {
  constexpr int kN = 8;                  // keys at a time; the next are on their way
  const int kh = h / L.group;
  const Row q = load_row(L.q.row(i, h), L.dim);
  Row acc = {{0.f, 0.f, 0.f, 0.f}};
  float m = -INFINITY, l = 0.f;
  Packed k[kN], v[kN], k1[kN], v1[kN];
  auto fetch = [&](int j) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      k1[n] = load_packed(L.k.row(min(j + n, i), kh), L.dim);
      v1[n] = load_packed(L.v.row(min(j + n, i), kh), L.dim);
    }
  };
  fetch(begin);
#pragma unroll 1
  for (int j = begin; j <= i; j += kN) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      k[n] = k1[n];
      v[n] = v1[n];
    }
    fetch(j + kN);
    float s[kN], mn = m;
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] = dot_part(q, unpack(k[n]));
    warp_sums(s);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      s[n] = j + n <= i ? L.scale * s[n] : -INFINITY;
      mn = fmaxf(mn, s[n]);
    }
    const float base = mn == -INFINITY ? 0.f : mn, f = __expf(m - base);
    l *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.v[e] *= f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float p = __expf(s[n] - base);
      l += p;
      axpy(acc, p, unpack(v[n]));
    }
    m = mn;
  }
  const float inv = 1.f / l;               // (l = 0, all scores -inf: NaN)
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.v[e] *= inv;
  return acc;
}

// Looks into output rows (bits of `bad`, from row r0 of the tile that starts at token row0)
// that are not finite although their weights are.  row_begin: of the lane's row.
static __device__ __noinline__ void mend_out(const AttentionLaunch& L, uint8_t* stage, int slabs,
                                             int h, int row0, int r0, int row_begin,
                                             unsigned int bad) {
  const int kh = h / L.group;
  unsigned int before = 0;                 // (rows that begin before the tile begin together)
  bool looked = false;
  while (bad) {
    const int src = __ffs(bad) - 1, r = r0 + src, i = row0 + r;
    bad &= bad - 1;
    const int begin = __shfl_sync(0xffffffffu, row_begin, src);
    unsigned int seen = bad_columns(L.v, kh, max(begin, row0), i + 1, L.dim);
    if (begin < row0) {
      if (!looked) before = bad_columns(L.v, kh, begin, row0, L.dim);
      looked = true;
      seen |= before;
    }
    if (__any_sync(0xffffffffu, bad_elements(stage, r, slabs) & ~seen))
      put_row(stage, r, out_row(L, h, i, begin), slabs);
  }
}

// Query gradient row i of head h.
static __device__ __noinline__ Row dq_row(const AttentionLaunch& L, int h, int i, int begin) {
  constexpr int kN = 4;
  const int kh = h / L.group;
  const Row q = load_row(L.q.row(i, h), L.dim);
  const Row g = load_row(L.dout.row(i, h), L.dim);
  float delta[1] = {dot_part(g, load_row(L.o.row(i, h), L.dim))};
  warp_sums(delta);
  const float lse = L.lse[static_cast<size_t>(h) * L.T + i];
  Row acc = {{0.f, 0.f, 0.f, 0.f}};
  Packed k[kN], v[kN], k1[kN], v1[kN];
  const __nv_bfloat16 *pk = L.k.row(begin, kh), *pv = L.v.row(begin, kh);
  auto fetch = [&](int j) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int dim = j + n <= i ? L.dim : 0;              // (past the last key: zeros)
      k1[n] = load_packed(pk, dim);
      v1[n] = load_packed(pv, dim);
      pk += L.k.ts;
      pv += L.v.ts;
    }
  };
  fetch(begin);
#pragma unroll 1
  for (int j = begin; j <= i; j += kN) {
    float s[2 * kN];                       // scores, dp
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      k[n] = k1[n];
      v[n] = v1[n];
    }
    fetch(j + kN);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      s[n] = dot_part(q, unpack(k[n]));
      s[kN + n] = dot_part(g, unpack(v[n]));
    }
    warp_sums(s);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float ds = __expf(L.scale * s[n] - lse) * (s[kN + n] - delta[0]);
      if (j + n <= i) axpy(acc, ds, unpack(k[n]));
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.v[e] *= L.scale;
  return acc;
}

// The same look for rows of dq, whose ds are finite: one of them stays as it is only where a
// visible key is not finite (and its weight 0).
static __device__ __noinline__ void mend_dq(const AttentionLaunch& L, uint8_t* stage, int slabs, int h,
                                            int row0, int r0, int row_begin, unsigned int bad) {
  const int kh = h / L.group;
  unsigned int before = 0;
  bool looked = false;
  while (bad) {
    const int src = __ffs(bad) - 1, r = r0 + src, i = row0 + r;
    bad &= bad - 1;
    const int begin = __shfl_sync(0xffffffffu, row_begin, src);
    unsigned int seen = bad_columns(L.k, kh, max(begin, row0), i + 1, L.dim);
    if (begin < row0) {
      if (!looked) before = bad_columns(L.k, kh, begin, row0, L.dim);
      looked = true;
      seen |= before;
    }
    if (__any_sync(0xffffffffu, bad_elements(stage, r, slabs) & ~seen))
      put_row(stage, r, dq_row(L, h, i, begin), slabs);
  }
}

// Columns of dv that a visible query's dout makes not finite, for key j of key head kh: the queries
// up to the end of the key's tile, and those behind it (the keys that see these end together).
struct Behind {
  bool looked = false;
  unsigned int columns = 0;
};
static __device__ __noinline__ unsigned int lost_columns(const AttentionLaunch& L, int kh, int key0,
                                                         int j, int end, Behind& behind) {
  const int edge = key0 + kBlock, h0 = kh * L.group, h1 = h0 + L.group;
  unsigned int lost = 0;
  for (int h = h0; h < h1; ++h) lost |= bad_columns(L.dout, h, j, min(end, edge), L.dim);
  if (end <= edge) return lost;
  if (!behind.looked)
    for (int h = h0; h < h1; ++h) behind.columns |= bad_columns(L.dout, h, edge, end, L.dim);
  behind.looked = true;
  return lost | behind.columns;
}

}  // namespace attn
}  // namespace muon
