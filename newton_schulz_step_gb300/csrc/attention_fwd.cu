// attention_fwd.cu -- causal attention over packed sequences with grouped key/value
// heads, forward, on the tensor cores.
//
// For the queries of a tile and the keys block by block:
//   S = Q K^T;  m' = max(m, rowmax S);  P = exp(scale (S - m'));  l = l f + rowsum P;
//   O = O f + P V  with f = exp(scale (m - m'));  at the end out = O / l,
//   lse = scale m + log l.
// The tokens are tiled as they lie, whatever the sequences: row i sees the keys
// begin(i) <= j <= i, so a tile of rows walks the key blocks from the first row's
// begin to its own diagonal block, and only blocks that hold a begin or the diagonal
// are masked.  No table of tiles is needed, and short sequences share tiles.
//
// A CTA takes 256 rows of one head as two tiles of 128.  While the compute warps turn
// one tile's S into P, the tensor cores run the other tile's products:
//   warps 0-3, 4-7  softmax of tile 0, 1 (a thread owns a row), then the epilogue
//   warp 8          TMA: Q once, then K and V blocks through a ring
//   warps 9, 10     MMA of tile 0, 1.  Heads of 128: per block  O += P V, then S of the next
//                   block, in turns, so that one tile's softmax falls on the other's
//                   products.  (One warp for both took 1500 cycles of waits and commits
//                   between its products, with the tensor cores idle; without turns the
//                   tiles fall into step.)  Heads of 64: S of the next block as soon as the
//                   softmax has read this one, then O += P V
//   warp 11         leaves its registers to the softmax
// (Two threads a row, with 16 warps for the softmax, were slower in an earlier form: 2204
// against 1623 us on 16384 tokens, 32/8 heads of 128 -- the exchange of the maxima costs
// more than the other warps hide.)
// TMEM: S of each tile (128 columns; P overwrites the first 64 as bf16 pairs, the A operand
// of P V, handed over in two halves), O of each tile.  tcgen05 ops of one thread run in
// order, so the commit that announces S of block b + 1 also says that P V of block b is
// done: O may be rescaled before P of block b + 1 is handed over.  O is rescaled only when
// the maximum grows by more than 2^8 (P stays below 2^8; fp32 sums and O hold that easily),
// so nearly never after the first blocks.  Heads of 64 leave room for P beside S: the next S
// is ready when its softmax begins, and a commit of its own says that P V is done.  8192
// tokens of 5 to 2400, 12 heads: 43.1 us instead of 45.6 with P over S.  (A third S instead,
// that either tile's next block takes: 42.9, but one sequence of 8192 tokens in 158 us
// instead of 154.)
// P is rounded to bf16, the tensor cores' input; l sums the unrounded values.
// What bounds it: with heads of 128 the tensor cores.  16384 tokens, 32/8 heads of 128: 1190 us
// for one call (1.85 PFLOP/s, as fast as a library product of that size), 1340 back to back
// under the power limit.  With heads of 64 a block's products take half the time, and its
// 16384 exponentials and the softmax's chain bound it; with few blocks a tile, the 5 us before
// a block's first product and after its last.
#include <climits>

#include "attention.cuh"

namespace muon {
namespace {

using namespace attn;

constexpr int kTiles = 2;
constexpr float kRescale = 8.f;        // log2 growth of the maximum that triggers a rescale

constexpr int kProducerWarp = 4 * kTiles, kMmaWarp = kProducerWarp + 1;   // and one a tile
constexpr int kThreads = 384;
constexpr uint32_t kMiscBytes = 512;

// Registers move from the warps that only issue work to those that compute: a block is
// launched with 168 a thread (64512), of which 4 warps keep kIssueRegs and 8 get
// kComputeRegs.  The issuing roles must fit kIssueRegs as compiled without the split (57):
// with 40 the compiler's allocation was seen to break (waits ran into their limit).
constexpr int kIssueRegs = 104, kComputeRegs = 200;
static_assert(128 * kIssueRegs + 256 * kComputeRegs == kThreads * 168,
              "no more registers than at launch");
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
}
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
}

template <int DP> struct Cfg {
  static constexpr uint32_t kTile = DP / 64 * kSlab;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr bool kOwnP = DP == 64;                    // P has columns of its own
  static constexpr uint32_t kOCol = kOwnP ? 384 : 256;
  static __device__ __forceinline__ uint32_t p_col(int t) { return kOwnP ? 256 + 64 * t : 128 * t; }
  static constexpr uint32_t kRing = kTiles * kTile;          // after Q
  static constexpr uint32_t kMisc = kRing + kStages * kTile;
  static constexpr uint32_t kSmem = kMisc + kMiscBytes;
};

struct Misc {
  uint64_t full[8], empty[8];
  uint64_t q_full[kTiles], s_full[kTiles], s_read[kTiles], p_full[kTiles][2], o_full[kTiles];
  uint64_t drain[kTiles], turn[kTiles];
  uint32_t tmem;
  int bad, skip;                       // abort flag; the workspace had failed before
  int first[kTiles], last[kTiles];     // begin of the first and last row of each tile
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc block");

__device__ __forceinline__ float row_max(const uint32_t (&s)[32]) {
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = max3(__uint_as_float(s[j]), __uint_as_float(s[j + 4]), __uint_as_float(s[j + 8]));
#pragma unroll
  for (int j = 12; j < 28; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = max3(x[e], __uint_as_float(s[j + e]), __uint_as_float(s[j + 4 + e]));
  const float a = max3(x[0], __uint_as_float(s[28]), __uint_as_float(s[29]));
  const float b = max3(x[1], __uint_as_float(s[30]), __uint_as_float(s[31]));
  return max3(a, b, fmaxf(x[2], x[3]));
}

__device__ __forceinline__ void tile_barrier(int t) {   // the four warps of a tile
  asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_fwd_kernel(const __grid_constant__ AttentionMaps M,
                         const __grid_constant__ AttentionLaunch L) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  Misc& X = *reinterpret_cast<Misc*>(sm + C::kMisc);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (warp == kProducerWarp && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&X.full[s], 1);
      ptx::mbar_init(&X.empty[s], kTiles);
    }
    for (int t = 0; t < kTiles; ++t) {
      ptx::mbar_init(&X.q_full[t], 1);
      ptx::mbar_init(&X.s_full[t], 1);
      ptx::mbar_init(&X.s_read[t], 4);
      ptx::mbar_init(&X.p_full[t][0], 4);
      ptx::mbar_init(&X.p_full[t][1], 4);
      ptx::mbar_init(&X.o_full[t], 1);
      ptx::mbar_init(&X.drain[t], 1);
      ptx::mbar_init(&X.turn[t], 1);
    }
    X.bad = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&M.q);
    ptx::prefetch_tmap(&M.k);
    ptx::prefetch_tmap(&M.v);
  }
  begin_after_prior();
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&X.tmem, 512);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    X.skip = ptx::status_set(L.status);
    if (!tiles_aligned(sm)) {
      atomicOr(L.status, kErrTimeoutAttention);
      X.skip = 1;
    }
  }

  // of one sequence, the last tiles hold the most keys: they go first
  const int rows = 128 * L.tiles, pairs = (L.T + rows - 1) / rows;
  const int h = static_cast<int>(blockIdx.x) % L.hq, kh = h / L.group;
  int row0 = (pairs - 1 - static_cast<int>(blockIdx.x) / L.hq) * rows;
  if (L.ranked)
    row0 = 128 * kTiles *
           ranked_tile(pairs, static_cast<int>(blockIdx.x) / L.hq, reinterpret_cast<int*>(sm),
                       [&](int i) {
                         const int r = 128 * kTiles * i;
                         return min(r + 128, L.T - 1) / kBlock - sequence_of(L, r).begin / kBlock;
                       });

  if (tid < 2 * kTiles) {
    const int r = row0 + 128 * (tid >> 1);
    const int i = (tid & 1) ? min(r + 127, L.T - 1) : r;
    const int b = r < L.T ? sequence_of(L, i).begin : 0;
    if (tid & 1) X.last[tid >> 1] = b;
    else X.first[tid >> 1] = b;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const Guard guard{&X.bad, L.status,
                    warp == kProducerWarp  ? kErrTimeoutProducer
                    : warp < kProducerWarp ? kErrTimeoutEpilogue
                                           : kErrTimeoutMma};

  // key blocks of each tile, [b0, b1), and of both
  int b0[kTiles], b1[kTiles], begin = INT_MAX, end = 0;   // (the same in every lane)
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int r = row0 + 128 * t;
    const bool used = t < L.tiles && r < L.T;
    b0[t] = used ? __shfl_sync(0xffffffffu, X.first[t], 0) / kBlock : 0;
    b1[t] = used ? r / kBlock + 1 : 0;
    if (used) {
      begin = min(begin, b0[t]);
      end = max(end, b1[t]);
    }
  }
  auto active = [&](int t, int b) { return b >= b0[t] && b < b1[t]; };

  const bool run = !X.skip;
  if (warp >= kProducerWarp) {
    registers_down();
    if (run && warp == kProducerWarp) {
      if (lane == 0) {
        int n = 0;                       // ring loads issued
        bool ok = true;
        auto load = [&](const CUtensorMap* map, int row) {
          const int s = n % C::kStages;
          if (n >= C::kStages)
            ok = ok && guard.wait_or_fail(&X.empty[s], (n / C::kStages - 1) & 1);
          if (!ok) return;
          load_tile<DP>(sm + C::kRing + s * C::kTile, map, kh, row, &X.full[s]);
          ++n;
        };
        for (int t = 0; t < kTiles; ++t)
          if (b1[t] > 0) load_tile<DP>(sm + t * C::kTile, &M.q, h, row0 + 128 * t, &X.q_full[t]);
        for (int b = begin; b < end && ok; ++b) {
          load(&M.k, b * kBlock);
          load(&M.v, b * kBlock);
        }
        if (!ok) {                       // copies in flight land before the CTA ends
          for (int t = 0; t < kTiles; ++t)
            if (b1[t] > 0) ptx::mbar_wait(&X.q_full[t], 0, nullptr, nullptr, kDrainNs);
          for (int i = n > C::kStages ? n - C::kStages : 0; i < n; ++i)
            ptx::mbar_wait(&X.full[i % C::kStages], (i / C::kStages) & 1, nullptr, nullptr,
                           kDrainNs);
        }
      }
    } else if (run && warp < kMmaWarp + kTiles) {
      const int t = warp - kMmaWarp;
      const int first = b0[t], last = b1[t];
      const uint32_t q = tile_address(sm) + t * C::kTile;
      const uint32_t ring = tile_address(sm) + C::kRing;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && guard.issue_wait(bar, parity);
        return ok;
      };
      // S of a block (the K tile has landed)
      auto scores = [&](int slot) {
        mma_heads<DP>(128 * t, q, ring + slot * C::kTile);
        ptx::mma_commit(&X.s_full[t]);
      };
      auto has = [&](int b) { return b >= first && b < last; };
      if constexpr (C::kOwnP) {
        auto load = [&](int n) {         // the slot of the ring's n-th load, which has landed
          wait(&X.full[n % C::kStages], (n / C::kStages) & 1);
          return n % C::kStages;
        };
        for (int b = begin - 1; b < end && ok; ++b) {
          if (b + 1 < end) {
            const int ks = load(2 * (b + 1 - begin));
            if (b + 1 == first && first < last) wait(&X.q_full[t], 0);
            if (has(b) && has(b + 1)) wait(&X.s_read[t], (b - first) & 1);
            ptx::tc_fence_after();
            if (ok && ptx::elect_one()) {
              if (has(b + 1)) scores(ks);
              ptx::mma_commit(&X.empty[ks]);
            }
            __syncwarp();
          }
          if (b < begin || !ok) continue;
          const int vs = load(2 * (b - begin) + 1);
          const bool mine = has(b);
          const uint32_t parity = (b - first) & 1, v = ring + vs * C::kTile;
          if (mine) {
            if (!wait(&X.p_full[t][0], parity)) break;
            ptx::tc_fence_after();
            if (ptx::elect_one())
              mma_rows<DP, 64, 32>(C::kOCol + DP * t, C::p_col(t), v, b > first);
            wait(&X.p_full[t][1], parity);
            ptx::tc_fence_after();
          }
          if (!ok) break;
          if (ptx::elect_one()) {
            if (mine) {
              mma_rows<DP, 64, 32>(C::kOCol + DP * t, C::p_col(t) + 32, v + 8192, true);
              ptx::mma_commit(&X.o_full[t]);
            }
            ptx::mma_commit(&X.empty[vs]);
          }
          __syncwarp();
        }
      } else {
        Ring<C::kStages> at;             // next slot of the ring
        auto take = [&] {
          const int s = at.slot;
          wait(&X.full[s], at.parity);
          at.next();
          return s;
        };
        if (begin < end) {
          const int ks = take();
          if (has(begin)) wait(&X.q_full[t], 0);
          if (ok && ptx::elect_one()) {
            if (has(begin)) scores(ks);
            ptx::mma_commit(&X.empty[ks]);
          }
        }
        for (int b = begin; b < end && ok; ++b) {
          // Waits for copies stand where nothing depends on them yet, and products that follow
          // one another go out together: every step of this warp between them costs the
          // tensor cores 100 cycles and more.
          const int vs = take();
          const int ks = b + 1 < end ? take() : -1;
          if (b + 1 == first && first < last) wait(&X.q_full[t], 0);
          const bool mine = has(b), next = has(b + 1);
          const uint32_t parity = (b - first) & 1, v = ring + vs * C::kTile;
          if (mine) wait(&X.p_full[t][0], parity);
          // the tiles take turns: tile 0 waits for tile 1's last block, tile 1 for this one
          if (!wait(&X.turn[t], ((b - begin) & 1) ^ (t == 0 ? 1 : 0))) break;
          if (mine) {
            ptx::tc_fence_after();
            if (ptx::elect_one())
              mma_rows<DP, 64, 32>(C::kOCol + DP * t, 128 * t, v, b > first);
            if (!wait(&X.p_full[t][1], parity)) break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            if (mine) mma_rows<DP, 64, 32>(C::kOCol + DP * t, 128 * t + 32, v + 8192, true);
            if (mine && b + 1 == last) ptx::mma_commit(&X.o_full[t]);
            if (next) scores(ks);
            ptx::mbar_arrive(&X.turn[t ^ 1]);
            ptx::mma_commit(&X.empty[vs]);
            if (ks >= 0) ptx::mma_commit(&X.empty[ks]);
          }
          __syncwarp();
        }
      }
      if (!ok) {                         // products in flight end before TMEM is freed
        if (ptx::elect_one()) ptx::mma_commit(&X.drain[t]);
        ptx::mbar_wait(&X.drain[t], 0, nullptr, nullptr, kDrainNs);
        __syncwarp();
      }
    }
  } else {
    registers_up();
    if (run) {
      const int t = warp >> 2, r = tid & 127, row = row0 + 128 * t + r;
      const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const uint32_t ts = lanes + 128 * t, tp = lanes + C::p_col(t);
      const uint32_t to = lanes + C::kOCol + DP * t;
      const int row_begin = row < L.T ? sequence_of(L, row).begin : row + 1;
      const int last_begin = X.last[t], first_block = b0[t], blocks_end = b1[t];
      const int used = tokens_in_use(L);
      const float c = L.scale * kLog2e;
      const uint64_t c2 = pair(c, c);
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int b = first_block; b < blocks_end; ++b) {
        const int k0 = b * kBlock;
        ok = guard.warp_wait(&X.s_full[t], (b - first_block) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[4][32];
        ptx::tmem_ld32x2_sync(ts, ts + 32, s[0], s[1]);
        ptx::tmem_ld32x2_sync(ts + 64, ts + 96, s[2], s[3]);
        if constexpr (C::kOwnP) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&X.s_read[t]);
        }
        bool clear = false;
        if (__builtin_expect(k0 < last_begin || b + 1 == blocks_end, 0)) {
          clear = k0 < X.first[0] || used < min(k0 + kBlock, L.T);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            hide(s[i], row_begin - k0 - 32 * i, row - k0 - 32 * i, 0xff800000u);
        }
        const float mb = fmaxf(fmaxf(row_max(s[0]), row_max(s[1])),
                               fmaxf(row_max(s[2]), row_max(s[3])));
        if (b == first_block) {
          m = mb;
        } else {
          if constexpr (C::kOwnP) {                    // P and O of the block before are free
            ok = guard.warp_wait(&X.o_full[t], (b - 1 - first_block) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
          }
          const bool grow = mb > m && !((mb - m) * c <= kRescale);
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
            const float f = grow ? ex2((m - mb) * c) : 1.f;
            if (grow) m = mb;
            l *= f;
#pragma unroll 1
            for (int i = 0; i < DP / 32; ++i) {
              uint32_t o[32];
              ptx::tmem_ld32_sync(to + 32 * i, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              ptx::tmem_st32(to + 32 * i, o);
            }
          }
        }
        if (__builtin_expect(clear, 0)) {
          // the block holds padding, or tokens that neither tile sees: clear their V
          const int n = 2 * (b - begin) + 1, slot = n % C::kStages;
          ok = guard.warp_wait(&X.full[slot], (n / C::kStages) & 1);
          if (!ok) break;
          if (k0 + r < X.first[0] || k0 + r >= used) zero_row<DP>(sm + C::kRing + slot * C::kTile, r);
          ptx::fence_proxy_async_smem();
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const uint64_t mc2 = pair(-mc, -mc);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 x = unpair(fma2(pair(__uint_as_float(s[i][2 * j]),
                                              __uint_as_float(s[i][2 * j + 1])), c2, mc2));
            const float2 y = make_float2(ex2(x.x), ex2(x.y));
            sum[j & 1] = add2(sum[j & 1], pair(y.x, y.y));
            p[j] = pack2(y.x, y.y);
          }
          ptx::tmem_st16(tp + 16 * i, p);
          if (i & 1) {                                 // half of P is ready for its product
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&X.p_full[t][i >> 1]);
          }
        }
        const float2 a = unpair(add2(sum[0], sum[1]));
        l += a.x + a.y;
      }
      if (ok && blocks_end > 0)
        ok = guard.warp_wait(&X.o_full[t], C::kOwnP ? (blocks_end - 1 - first_block) & 1 : 0);
      if (ok && blocks_end > 0) {
        ptx::tc_fence_after();
        // Q of this tile has been read for the last time: out goes through its place
        uint8_t* stage = sm + t * C::kTile;
        // A row without keys (padding) is 0, -inf.  One whose visible scores are all -inf has
        // l = 0 too, and is NaN by the definition: 0 times 1 / 0 here, and lse in its place.
        const bool keys = row_begin <= row;
        const float inv = 1.f / l;
        float test = 0.f;                              // NaN if an element is not finite
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          uint32_t o[32];
          ptx::tmem_ld32_sync(to + 32 * i, o);
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            f[j] = keys ? __uint_as_float(o[j]) * inv : 0.f;
            test = fmaf(f[j], 0.f, test);
          }
          store_row32(stage, r, 4 * i, f);
        }
        if (row < L.T)
          L.lse[static_cast<size_t>(h) * L.T + row] =
              !keys ? -INFINITY : l == 0.f ? NAN : m * L.scale + __logf(l);
        __syncwarp();
        // (a row whose l is NaN or 0 is NaN throughout)
        const unsigned int bad = __ballot_sync(0xffffffffu, row < L.T && test != 0.f && l > 0.f);
        if (bad) mend_out(L, stage, DP / 64, h, row0 + 128 * t, r - lane, row_begin, bad);
        ptx::fence_proxy_async_smem();
      }
      if (blocks_end > 0) {
        tile_barrier(t);                               // (reached by every thread of the tile)
        if (ok && r == 0 && !X.bad) {
#pragma unroll
          for (int i = 0; i < DP / 64; ++i)
            ptx::tma_store_3d(&M.out, 64 * i, h, row0 + 128 * t, sm + t * C::kTile + i * kSlab);
          ptx::bulk_commit();
          ptx::bulk_wait_read<0>();
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(X.tmem, 512);
  }
}

template <int DP>
cudaError_t launch(const AttentionMaps& m, AttentionLaunch& l, int sms, cudaStream_t s) {
  static_assert(Cfg<DP>::kSmem <= 232448, "shared memory");
  // a tile a CTA while that takes no second wave (2048 tokens, 8 heads of 64: 26 us
  // instead of 28; 1024: 18 instead of 20)
  l.tiles = (l.T + 127) / 128 * l.hq <= sms ? 1 : kTiles;
  const int pairs = (l.T + 128 * l.tiles - 1) / (128 * l.tiles);
  l.ranked = rank_tiles(l.n_seqs, pairs, l.hq, sms);
  return launch_behind(attention_fwd_kernel<DP>, pairs * l.hq, kThreads, Cfg<DP>::kSmem, m, l, s);
}

}  // namespace

cudaError_t launch_attention(const AttentionMaps& m, AttentionLaunch l, int sms, cudaStream_t s) {
  return l.dim <= 64 ? launch<64>(m, l, sms, s) : launch<128>(m, l, sms, s);
}

}  // namespace muon
