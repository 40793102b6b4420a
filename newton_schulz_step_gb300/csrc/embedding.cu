// embedding.cu -- rows of a token table, scaled, and the table's gradient
//
//   out[t] = scale table[id_t],     d table[v] = scale sum over {t : id_t = v} of dout[t]
//
// The lookup is one read and one write of each token's row.  The gradient writes every row
// of the table, zeros too, and reads dout once; each row's sum has a fixed order, by tokens
// sorted by id (stable, so ascending in a row):
//
//   embedding_sort_kernel   one cluster of 8 CTAs sorts the tokens (radix, up to 10 bits a
//                           pass) while the other CTAs of the launch clear the gradient: the
//                           sort has 8 SMs' worth of work, the clearing is bound by HBM
//   embedding_sum_kernel    a warp takes 32 sorted positions and 256 columns, adds the rows
//                           of a run of equal ids in registers and stores the run; what
//                           begins or ends outside of the 32 goes to the workspace
//   embedding_join_kernel   runs that cross a border: their pieces, in order
//
// Runs are cut by position, not by id, so that a token that makes up a tenth of a text is
// shared by many warps.  Rows that a run fills are written twice (cleared, then stored); they
// are few against the table, and still in L2.
//
// 32768 tokens of a text's frequencies, 50257 rows of 768: lookup 11.9 us; gradient 48 us for
// 205 MB (4.2 TB/s) back to back; each launch by itself with cold caches: clearing and sort 27
// (the sort without clearing 22), sums 15, joins 10.  With digits' equals found by __match_any_sync,
// items read again for their placing, and the joins of a token's 48 pieces by one warp it
// was 96.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 elements as stored.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack(a, v); }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
// -1 for an id outside the table.
__device__ __forceinline__ int id_at(const void* ids, bool wide, int t, int rows) {
  const long long v = wide ? __ldg(static_cast<const long long*>(ids) + t)
                           : static_cast<long long>(__ldg(static_cast<const int*>(ids) + t));
  return v >= 0 && v < rows ? static_cast<int>(v) : -1;
}

// ------------------------------------------------------------ lookup
// A warp takes a token's row, kAt vectors a lane in flight; the next token's id travels
// with them.
constexpr int kAt = 4;
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ EmbeddingLaunch L) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int stride = gridDim.x * (kThreads / 32);
  const int vecs = L.dim >> 3;
  int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  int id = t < L.tokens ? id_at(L.ids, L.wide, t, L.rows) : -1;
  for (; t < L.tokens; t += stride) {
    const int next = t + stride < L.tokens ? id_at(L.ids, L.wide, t + stride, L.rows) : -1;
    const T* const row = static_cast<const T*>(L.table) + max(id, 0) * L.table_stride;
    O* const out = static_cast<O*>(L.out) + t * L.out_stride;
    const float scale = id < 0 ? __int_as_float(0x7fffffff) : L.scale;
    for (int c = lane; c < vecs; c += 32 * kAt) {
      float v[kAt][8];
#pragma unroll
      for (int i = 0; i < kAt; ++i)
        if (c + 32 * i < vecs) load8(row + 8 * (c + 32 * i), v[i]);
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        if (c + 32 * i >= vecs) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= scale;
        store8(out + 8 * (c + 32 * i), v[i]);
      }
    }
    id = next;
  }
}

// ------------------------------------------------------------ sort, and zeros
constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 1024;
constexpr int kSortSmem = (kSortWarps * kMaxBins + 2 * kMaxBins + 64) * 4;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Lanes of the warp that hold the digit d of this one: a ballot a bit.  (__match_any_sync took
// about six times as long for digits of 8 bits.)  Lanes that are not live hold none.
__device__ __forceinline__ uint32_t equal_lanes(uint32_t d, int bits, bool live) {
  uint32_t same = __ballot_sync(0xffffffffu, live);
  for (int b = 0; b < bits; ++b) {
    const uint32_t ones = __ballot_sync(0xffffffffu, d >> b & 1u);
    same &= d >> b & 1u ? ones : ~ones;
  }
  return same;
}

constexpr int kRounds = 8;             // items of a lane at a time
struct Batch {
  uint32_t key[kRounds], off[kRounds];
  uint32_t live;                       // bit r: item r is there
};
// Adds a batch's digits to the warp's counters; off: place of an item among the warp's items
// of its digit.
__device__ __forceinline__ void rank_batch(Batch& b, uint32_t* mine, int shift, int bits) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool live = b.live >> r & 1u;
    if (!__any_sync(0xffffffffu, live)) continue;
    const uint32_t d = b.key[r] >> shift & ((1u << bits) - 1u);
    const uint32_t same = equal_lanes(d, bits, live);
    const uint32_t rank = __popc(same & ((1u << lane) - 1u));
    if (live) b.off[r] = mine[d] + rank;
    __syncwarp();
    if (live && rank == 0u) mine[d] += __popc(same);
    __syncwarp();
  }
}

// Sorts (id, token) by `passes` digits of `bits` bits, least first; tokens whose id is outside
// the table are dropped, and their number is left in *L.count.  CTA r has the r-th contiguous
// part of the items, a warp a contiguous part of it, and each pass keeps equal digits in order:
// counts a warp, a digit's place from the counts of smaller digits, earlier CTAs and earlier
// warps, and an item's place among its warp's.  A warp's items stay in registers between the
// count and the placing while they are kRounds a lane (up to 65536 tokens); more are read and
// ranked again.  8 SMs take 22 us for 32768 tokens in two passes of 8 bits.
__device__ void sort_tokens(const EmbeddingLaunch& L, uint32_t* smem) {
  uint32_t* const cnt = smem;                              // [warps][bins]
  uint32_t* const total = smem + kSortWarps * kMaxBins;    // [bins], read by the other CTAs
  uint32_t* const base = total + kMaxBins;                 // [bins]
  uint32_t* const scan = base + kMaxBins;                  // [warps + 1]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const uint32_t rank = ptx::cluster_ctarank();
  const int bins = 1 << L.bits;
  uint32_t* const mine = cnt + warp * kMaxBins;
  int items = L.tokens;
  for (int pass = 0; pass < L.passes; ++pass) {
    // the last pass ends in keys / order [0]
    const int to = (L.passes - 1 - pass) & 1, from = to ^ 1;
    const int shift = pass * L.bits;
    // whole rounds of 32 a warp
    constexpr int kPer = kSortCtas * kSortWarps * 32;
    const int per_warp = static_cast<int>((static_cast<long long>(items) + kPer - 1) / kPer) * 32;
    const long long begin = (static_cast<long long>(rank) * kSortWarps + warp) * per_warp;
    const int i0 = static_cast<int>(min(begin, static_cast<long long>(items)));
    const int i1 = static_cast<int>(min(begin + per_warp, static_cast<long long>(items)));
    const bool one_batch = per_warp <= 32 * kRounds;
    Batch b;
    auto load = [&](int i) {           // items i + 32 r + lane
      b.live = 0u;
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int at = i + 32 * r + lane;
        b.key[r] = 0u;
        bool live = at < i1;
        if (live) {
          if (pass > 0) {
            b.key[r] = __ldcg(L.keys[from] + at);
          } else {
            const int id = id_at(L.ids, L.wide, at, L.rows);
            live = id >= 0;
            b.key[r] = static_cast<uint32_t>(id);
          }
        }
        b.live |= static_cast<uint32_t>(live) << r;
      }
    };
    load(i0);
    for (int k = lane; k < bins; k += 32) mine[k] = 0u;
    __syncwarp();
    rank_batch(b, mine, shift, L.bits);
    for (long long i = static_cast<long long>(i0) + 32 * kRounds; i < i1; i += 32 * kRounds) {
      load(static_cast<int>(i));
      rank_batch(b, mine, shift, L.bits);
    }
    __syncthreads();
    // a thread a digit: places of the warps, the CTA's total
    if (tid < bins) {
      uint32_t run = 0u;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = cnt[w * kMaxBins + tid];
        cnt[w * kMaxBins + tid] = run;
        run += n;
      }
      total[tid] = run;
    }
    ptx::cluster_sync();
    uint32_t before = 0u, all = 0u;
    if (tid < bins) {
      const uint32_t at = ptx::smem_u32(total + tid);
#pragma unroll
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        const uint32_t n = ld_cluster_u32(ptx::mapa_shared(at, r));
        if (r < rank) before += n;
        all += n;
      }
    }
    // exclusive scan of the digits' totals over the block
    uint32_t x = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    if (warp == 0) {
      const uint32_t own = scan[lane];
      uint32_t y = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      scan[lane] = y - own;
      if (lane == 31) scan[kSortWarps] = y;
    }
    __syncthreads();
    if (tid < bins) base[tid] = scan[warp] + x - all + before;
    items = static_cast<int>(scan[kSortWarps]);            // (less the dropped ones)
    __syncthreads();
    auto place = [&](int i, bool ranked) {
      uint32_t token[kRounds];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        token[r] = static_cast<uint32_t>(i + 32 * r + lane);
        if (pass > 0 && (b.live >> r & 1u)) token[r] = __ldcg(L.order[from] + token[r]);
      }
      if (!ranked) rank_batch(b, mine, shift, L.bits);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (!(b.live >> r & 1u)) continue;
        const uint32_t d = b.key[r] >> shift & (bins - 1);
        const uint32_t at = base[d] + b.off[r] + (ranked ? mine[d] : 0u);
        __stcg(L.keys[to] + at, b.key[r]);
        __stcg(L.order[to] + at, token[r]);
      }
    };
    if (one_batch) {
      place(i0, true);
    } else {
      for (long long i = i0; i < i1; i += 32 * kRounds) {
        load(static_cast<int>(i));
        place(static_cast<int>(i), false);
      }
    }
    // the other CTAs' stores of this pass are read by the next, and `total` is free again
    __threadfence();
    ptx::cluster_sync();
  }
  if (rank == 0 && tid == 0) __stcg(L.count, static_cast<uint32_t>(items));
}

__global__ void __launch_bounds__(kSortThreads, 1)
    embedding_sort_kernel(const __grid_constant__ EmbeddingLaunch L) {
  extern __shared__ uint32_t s_sort[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;      // (the same word for every CTA of the cluster)
  if (blockIdx.x < kSortCtas) {
    sort_tokens(L, s_sort);
    return;
  }
  // zeros, 16 bytes a store
  const int unit = L.out_bf16 ? 8 : 4;                    // elements
  const long long size = L.out_bf16 ? 2 : 4;
  const long long per_row = L.dim / unit;
  const long long total = per_row * L.rows;
  const long long step = static_cast<long long>(gridDim.x - kSortCtas) * kSortThreads;
  uint8_t* const out = static_cast<uint8_t*>(L.out);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  long long i = static_cast<long long>(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x;
  if (L.out_stride == L.dim) {
#pragma unroll 4
    for (; i < total; i += step) *reinterpret_cast<uint4*>(out + i * 16) = zero;
  } else {
    for (; i < total; i += step) {
      const long long r = i / per_row;
      *reinterpret_cast<uint4*>(out + (r * L.out_stride + (i - r * per_row) * unit) * size) = zero;
    }
  }
}

// ------------------------------------------------------------ sums
template <typename O>
__device__ __forceinline__ void store_row(const EmbeddingLaunch& L, uint32_t id, int c,
                                          float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= L.scale;
  if (id < static_cast<uint32_t>(L.rows)) store8(static_cast<O*>(L.out) + id * L.out_stride + c, v);
}

constexpr int kChunk = 32;             // sorted positions of a warp
template <typename G> constexpr int kFlight = 16 / sizeof(G);   // rows of a warp in flight
template <typename G, typename O>
__global__ void __launch_bounds__(kThreads, 3)
    embedding_sum_kernel(const __grid_constant__ EmbeddingLaunch L) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int groups = (L.dim + 255) / 256;
  const long long task = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int chunk = static_cast<int>(task / groups);
  const int c = static_cast<int>(task - static_cast<long long>(chunk) * groups) * 256 + lane * 8;
  const long long i0 = static_cast<long long>(chunk) * kChunk;
  // everything that the rows depend on in one trip: the lists are allocated to L.tokens, of
  // which the first *L.count positions are sorted tokens
  const bool there = i0 + lane < L.tokens;
  const bool failed = ptx::status_set(L.status);
  const long long items = min(__ldcg(L.count), static_cast<uint32_t>(L.tokens));
  uint32_t key = there ? __ldcg(L.keys[0] + i0 + lane) : 0u;
  uint32_t token = there ? __ldcg(L.order[0] + i0 + lane) : 0u;
  const uint32_t before = i0 > 0 ? __ldcg(L.keys[0] + i0 - 1) : 0u;
  const uint32_t after = i0 + kChunk < L.tokens ? __ldcg(L.keys[0] + i0 + kChunk) : 0u;
  if (failed || i0 >= items) return;
  const int n = static_cast<int>(min(static_cast<long long>(kChunk), items - i0));
  // (a list that another call wrote into, against the contract, reaches no other memory)
  if (lane >= n || token >= static_cast<uint32_t>(L.tokens)) token = 0u;
  // bit i: a run begins at position i; the run at position 0 may have begun earlier
  const uint32_t prev = __shfl_up_sync(0xffffffffu, key, 1);
  const bool head_open = i0 > 0 && before == __shfl_sync(0xffffffffu, key, 0);
  const bool tail_open = i0 + kChunk < items && after == __shfl_sync(0xffffffffu, key, kChunk - 1);
  const uint32_t begins = __ballot_sync(0xffffffffu, lane < n && (lane == 0 || key != prev));
  const bool on = c < L.dim;
  const G* const column = static_cast<const G*>(L.dout) + (on ? c : 0);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  int begin = 0;
#pragma unroll 1
  for (int p = 0; p < n; p += kFlight<G>) {
    Raw<G> raw[kFlight<G>];
#pragma unroll
    for (int k = 0; k < kFlight<G>; ++k) {
      // (positions past the last read token 0's row and are not added)
      const uint32_t t = __shfl_sync(0xffffffffu, token, (p + k) & 31);
      raw[k].load(column + t * L.dout_stride);
    }
#pragma unroll
    for (int k = 0; k < kFlight<G>; ++k) {
      const int i = p + k;
      if (i >= n) break;
      if (begins >> i & 1u) {
        begin = i;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      }
      float v[8];
      raw[k].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
      if (i + 1 < n && !(begins >> (i + 1) & 1u)) continue;   // the run goes on in this chunk
      const uint32_t id = __shfl_sync(0xffffffffu, key, i);
      if (!on) continue;
      const bool from_before = begin == 0 && head_open;
      const bool goes_on = i + 1 == n && tail_open;
      if (from_before || goes_on) {
        // [chunk][0]: of a run that began earlier; [1]: of one that begins here
        store8(L.parts + (static_cast<size_t>(chunk) * 2 + (from_before ? 0 : 1)) * L.dim + c, acc);
      } else {
        store_row<O>(L, id, c, acc);
      }
    }
  }
}

// A run that begins in a chunk and goes on: its piece there, then those of the chunks after.
// A warp adds a few pieces by itself; the pieces of longer runs (a token that makes up much of
// a text) are shared by the block's warps, every eighth one each, and the warps' sums added in
// order.
constexpr int kAlone = 8;              // pieces
template <typename O>
__global__ void __launch_bounds__(kThreads)
    embedding_join_kernel(const __grid_constant__ EmbeddingLaunch L) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float s_sum[kWarps][256];
  __shared__ int s_reach[kWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk0 = blockIdx.x * kWarps;                  // a warp a chunk, 256 columns a block
  const int c = blockIdx.y * 256 + lane * 8;
  const int chunk = chunk0 + warp;
  const long long first = static_cast<long long>(chunk) * kChunk, last = first + kChunk - 1;
  const bool inside = last + 1 < L.tokens;
  const bool failed = ptx::status_set(L.status);
  const long long items = min(__ldcg(L.count), static_cast<uint32_t>(L.tokens));
  const uint32_t id = inside ? __ldcg(L.keys[0] + last) : 0u;
  const uint32_t after = inside ? __ldcg(L.keys[0] + last + 1) : 0u;
  const uint32_t before = inside && first > 0 ? __ldcg(L.keys[0] + first - 1) : 0u;
  // it goes on, and did not begin earlier
  const bool open = !failed && last + 1 < items && id == after && !(first > 0 && before == id);
  // chunks after this one that the run reaches: all up to the first that it does not fill
  int reach = 0;
  for (int k = chunk + 1; open; k += 32) {
    const long long end = (static_cast<long long>(k) + lane) * kChunk + kChunk - 1;
    const bool through = end + 1 < items && __ldcg(L.keys[0] + end) == id &&
                         __ldcg(L.keys[0] + end + 1) == id;
    const uint32_t stop = __ballot_sync(0xffffffffu, !through);
    if (stop != 0u) {
      reach = k - chunk + __ffs(stop) - 1;
      break;
    }
  }
  const bool on = c < L.dim;
  const float* const column = L.parts + (on ? c : 0);
  auto piece = [&](int k, float (&v)[8]) {                 // k pieces after a chunk's: [k][0]
    load8(column + static_cast<size_t>(k) * 2 * L.dim, v);
  };
  if (open && reach <= kAlone) {
    float acc[8], v[8];
    load8(column + (static_cast<size_t>(chunk) * 2 + 1) * L.dim, acc);
#pragma unroll 4
    for (int k = 1; k <= reach; ++k) {
      piece(chunk + k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
    if (on) store_row<O>(L, id, c, acc);
  }
  if (lane == 0) s_reach[warp] = open && reach > kAlone ? reach : 0;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    const int far = s_reach[w];
    if (far == 0) continue;                                // (the same for every thread)
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if (warp == 0) load8(column + (static_cast<size_t>(chunk0 + w) * 2 + 1) * L.dim, acc);
#pragma unroll 8
    for (int k = 1 + warp; k <= far; k += kWarps) {
      float v[8];
      piece(chunk0 + w + k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
    store8(&s_sum[warp][lane * 8], acc);
    __syncthreads();
    if (warp == w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        float v[8];
        load8(&s_sum[i][lane * 8], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[j];
      }
      if (on) store_row<O>(L, id, c, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ launchers
template <typename K>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, int cluster,
                             cudaStream_t s, const EmbeddingLaunch& l) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, l);
}

// Clusters of the sort that fit on the current device at once, asked once a device.
cudaError_t sort_clusters(int sms, int* out) {
  static int cache[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (cache[dev] == 0) {
    e = cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kSortCtas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(kSortCtas * (sms / kSortCtas));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, embedding_sort_kernel, &cfg);
    if (e != cudaSuccess) return e;
    cache[dev] = n < 1 ? 1 : n;
  }
  *out = cache[dev];
  return cudaSuccess;
}

long long warp_tasks(const EmbeddingLaunch& l) {
  return 1ll * ((l.tokens + kChunk - 1) / kChunk) * ((l.dim + 255) / 256);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingLaunch& l, bool table_bf16, int sms, cudaStream_t s) {
  constexpr int kPer = kThreads / 32;
  const dim3 blocks(static_cast<unsigned>(
      std::min<long long>((1ll * l.tokens + kPer - 1) / kPer, 8ll * sms)));
  using B = __nv_bfloat16;
  if (table_bf16)
    return l.out_bf16 ? launch_dependent(embedding_kernel<B, B>, blocks, kThreads, 0, 1, s, l)
                      : launch_dependent(embedding_kernel<B, float>, blocks, kThreads, 0, 1, s, l);
  return l.out_bf16 ? launch_dependent(embedding_kernel<float, B>, blocks, kThreads, 0, 1, s, l)
                    : launch_dependent(embedding_kernel<float, float>, blocks, kThreads, 0, 1, s, l);
}

cudaError_t launch_embedding_sort(EmbeddingLaunch l, int sms, cudaStream_t s) {
  // passes of at most 10 bits that cover 0..rows - 1
  int bits = 1;
  while (bits < 31 && ((l.rows - 1) >> bits) != 0) ++bits;
  l.passes = (bits + 9) / 10;
  l.bits = (bits + l.passes - 1) / l.passes;
  int fit = 0;
  const cudaError_t e = sort_clusters(sms, &fit);
  if (e != cudaSuccess) return e;
  // the sort's cluster, and clusters that clear: those that fit beside it (a second wave would
  // take as long as the first), at least one
  const long long bytes = 1ll * l.rows * l.dim * (l.out_bf16 ? 2 : 4);
  const long long want = bytes / (kSortCtas * kSortThreads * 64) + 1;
  const long long clear = std::max(1ll, std::min<long long>(fit - 1, want));
  return launch_dependent(embedding_sort_kernel,
                          dim3(static_cast<unsigned>(kSortCtas * (1 + clear))), kSortThreads,
                          kSortSmem, kSortCtas, s, l);
}

cudaError_t launch_embedding_sum(const EmbeddingLaunch& l, bool dout_bf16, cudaStream_t s) {
  const dim3 blocks(static_cast<unsigned>((warp_tasks(l) + kThreads / 32 - 1) / (kThreads / 32)));
  using B = __nv_bfloat16;
  auto go = [&](auto kernel) { return launch_dependent(kernel, blocks, kThreads, 0, 1, s, l); };
  if (dout_bf16)
    return l.out_bf16 ? go(embedding_sum_kernel<B, B>) : go(embedding_sum_kernel<B, float>);
  return l.out_bf16 ? go(embedding_sum_kernel<float, B>) : go(embedding_sum_kernel<float, float>);
}

cudaError_t launch_embedding_join(const EmbeddingLaunch& l, cudaStream_t s) {
  constexpr int kPer = kChunk * (kThreads / 32);
  const dim3 grid(static_cast<unsigned>((1ll * l.tokens + kPer - 1) / kPer), (l.dim + 255) / 256);
  return l.out_bf16
             ? launch_dependent(embedding_join_kernel<__nv_bfloat16>, grid, kThreads, 0, 1, s, l)
             : launch_dependent(embedding_join_kernel<float>, grid, kThreads, 0, 1, s, l);
}

size_t embedding_parts(int tokens, int dim) {
  const size_t chunks = (static_cast<size_t>(tokens) + kChunk - 1) / kChunk;
  return chunks > 1 ? chunks * 2 * dim : 0;
}

}  // namespace muon
