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
// A CTA takes 256 rows of one head as two tiles of 128.  While a warpgroup turns one
// tile's S into P, the tensor cores run the other tile's products:
//   warps 0-3, 4-7  softmax of tile 0, 1 (a thread owns a row), then the epilogue
//   warp 8          TMA: Q once, then K and V blocks through a ring
//   warp 9          MMA: per block and tile  O += P V, then S of the next block
//   warps 10, 11    leave their registers to the softmax
// TMEM: S of each tile (128 columns; P overwrites its first 64 as bf16 pairs, the A
// operand of P V), O of each tile.  tcgen05 ops of one thread run in order, so the
// commit that announces S of block b + 1 also says that P V of block b is done: O may
// be rescaled before P of block b + 1 is handed over.  O is rescaled only when the
// maximum grows by more than 2^8 (P stays below 2^8; fp32 sums and O hold that
// easily), so nearly never after the first blocks.
// P is rounded to bf16, the tensor cores' input; l sums the unrounded values.
#include <climits>

#include "attention.cuh"

namespace muon {
namespace {

using namespace attn;

constexpr int kTiles = 2;
constexpr int kProducerWarp = 4 * kTiles, kMmaWarp = kProducerWarp + 1;
constexpr float kRescale = 8.f;        // log2 growth of the maximum that triggers a rescale

template <int DP> struct Cfg {
  static constexpr uint32_t kTile = DP / 64 * kSlab;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr uint32_t kRing = kTiles * kTile;          // after Q
  static constexpr uint32_t kMisc = kRing + kStages * kTile;
  static constexpr uint32_t kSmem = kMisc + 512 + 1024;
};

struct Misc {
  uint64_t full[8], empty[8];
  uint64_t q_full[kTiles], s_full[kTiles], p_full[kTiles], o_full[kTiles];
  uint64_t drain;
  uint32_t tmem;
  int bad, skip;                       // abort flag; the workspace had failed before
  int first[kTiles], last[kTiles];     // begin of the first and last row of each tile
};
static_assert(sizeof(Misc) <= 512, "misc block");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_fwd_kernel(const __grid_constant__ AttentionMaps M,
                         const __grid_constant__ AttentionLaunch L) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  Misc& X = *reinterpret_cast<Misc*>(sm + C::kMisc);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // the last tiles hold the most keys: they go first
  const int pairs = (L.T + 128 * kTiles - 1) / (128 * kTiles);
  const int h = static_cast<int>(blockIdx.x) % L.hq;
  const int row0 = (pairs - 1 - static_cast<int>(blockIdx.x) / L.hq) * (128 * kTiles);
  const int kh = h / L.group;

  if (tid < 2 * kTiles) {
    const int r = row0 + 128 * (tid >> 1);
    const int i = (tid & 1) ? min(r + 127, L.T - 1) : r;
    const int b = r < L.T ? sequence_of(L, i).begin : 0;
    if (tid & 1) X.last[tid >> 1] = b;
    else X.first[tid >> 1] = b;
  }
  if (warp == kProducerWarp && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&X.full[s], 1);
      ptx::mbar_init(&X.empty[s], 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      ptx::mbar_init(&X.q_full[t], 1);
      ptx::mbar_init(&X.s_full[t], 1);
      ptx::mbar_init(&X.p_full[t], 4);
      ptx::mbar_init(&X.o_full[t], 1);
    }
    ptx::mbar_init(&X.drain, 1);
    X.bad = 0;
    X.skip = ptx::status_set(L.status);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&M.q);
    ptx::prefetch_tmap(&M.k);
    ptx::prefetch_tmap(&M.v);
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&X.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const Guard guard{&X.bad, L.status,
                    warp == kProducerWarp ? kErrTimeoutProducer
                    : warp == kMmaWarp    ? kErrTimeoutMma
                                          : kErrTimeoutEpilogue};

  // key blocks of each tile, [b0, b1), and of both
  int b0[kTiles], b1[kTiles], begin = INT_MAX, end = 0;   // (the same in every lane)
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int r = row0 + 128 * t;
    b0[t] = __shfl_sync(0xffffffffu, X.first[t], 0) / kBlock;
    b1[t] = r < L.T ? r / kBlock + 1 : 0;
    if (r < L.T) {
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
    } else if (run && warp == kMmaWarp) {
      const uint32_t sq = ptx::smem_u32(sm), ring = sq + C::kRing;
      Ring<C::kStages> at;               // next slot of the ring
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && guard.warp_wait(bar, parity);
        if (ok) ptx::tc_fence_after();
        return ok;
      };
      auto take = [&] {
        const int s = at.slot;
        wait(&X.full[s], at.parity);
        at.next();
        return s;
      };
      auto scores = [&](int t, int b, int slot) {
        if (b == b0[t] && !wait(&X.q_full[t], 0)) return;
        if (ptx::elect_one()) {
          mma_heads<DP>(128 * t, sq + t * C::kTile, ring + slot * C::kTile);
          ptx::mma_commit(&X.s_full[t]);
        }
      };
      int ks = take();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (ok && active(t, begin)) scores(t, begin, ks);
      if (ok && ptx::elect_one()) ptx::mma_commit(&X.empty[ks]);
      for (int b = begin; b < end && ok; ++b) {
        const int vs = take();
        ks = b + 1 < end ? take() : -1;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (ok && active(t, b) && wait(&X.p_full[t], (b - b0[t]) & 1)) {
            if (ptx::elect_one()) {
              mma_rows<DP>(128 * kTiles + DP * t, [t](int i) { return 128u * t + 8 * i; },
                           ring + vs * C::kTile, b > b0[t]);
              if (b + 1 == b1[t]) ptx::mma_commit(&X.o_full[t]);
            }
          }
          if (ok && active(t, b + 1)) scores(t, b + 1, ks);
        }
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::mma_commit(&X.empty[vs]);
          if (ks >= 0) ptx::mma_commit(&X.empty[ks]);
        }
      }
      if (!ok) {                         // products in flight end before TMEM is freed
        if (ptx::elect_one()) ptx::mma_commit(&X.drain);
        ptx::mbar_wait(&X.drain, 0, nullptr, nullptr, kDrainNs);
        __syncwarp();
      }
    }
  } else {
    registers_up();
    if (run) {
      const int t = warp >> 2, r = tid & 127;
      const int row = row0 + 128 * t + r;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = lanes + 128 * t, to = lanes + 128 * kTiles + DP * t;
      const int row_begin = row < L.T ? sequence_of(L, row).begin : row + 1;
      const int last_begin = X.last[t];
      const int used = tokens_in_use(L);
      const float c = L.scale * kLog2e;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int b = b0[t]; b < b1[t]; ++b) {
        ok = guard.warp_wait(&X.s_full[t], (b - b0[t]) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[4][32];
        ptx::tmem_ld128_sync(ts, s);
        const int k0 = b * kBlock;
        if (k0 < last_begin || b + 1 == b1[t]) {
          const int lo = row_begin - k0, hi = row - k0;      // visible columns
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * i + j < lo || 32 * i + j > hi) s[i][j] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
          for (int j = 1; j < 32; ++j) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][j]));
        }
        const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (b == b0[t]) {
          m = mb;
        } else {
          const bool grow = mb > m && !((mb - m) * c <= kRescale);
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? ex2((m - mb) * c) : 1.f;
            if (grow) m = mb;
            l *= f;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
              uint32_t o[32];
              ptx::tmem_ld32_sync(to + 32 * i, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              ptx::tmem_st32(to + 32 * i, o);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = ex2(fmaf(__uint_as_float(s[i][2 * j]), c, -mc));
            const float y = ex2(fmaf(__uint_as_float(s[i][2 * j + 1]), c, -mc));
            sum[j & 3] += x + y;
            p[j] = pack2(x, y);
          }
          ptx::tmem_st16(ts + 16 * i, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (used < min(k0 + kBlock, L.T)) {            // the block holds padding: clear its V
          const int n = 2 * (b - begin) + 1, slot = n % C::kStages;
          ok = guard.warp_wait(&X.full[slot], (n / C::kStages) & 1);
          if (!ok) break;
          if (k0 + r >= used) zero_row<DP>(sm + C::kRing + slot * C::kTile, r);
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&X.p_full[t]);
      }
      if (ok && b1[t] > 0) {
        ok = guard.warp_wait(&X.o_full[t], 0);
        ptx::tc_fence_after();
        if (ok) {
          // Q of this tile has been read for the last time: out goes through its place
          uint8_t* stage = sm + t * C::kTile;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          float test = 0.f;                            // NaN if an element is not finite
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) {
            uint32_t o[32];
            ptx::tmem_ld32_sync(to + 32 * i, o);
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              f[j] = l == 0.f ? 0.f : __uint_as_float(o[j]) * inv;
              test = fmaf(f[j], 0.f, test);
            }
            store_row32(stage, r, 4 * i, f);
          }
          if (row < L.T)
            L.lse[static_cast<size_t>(h) * L.T + row] =
                l == 0.f ? -INFINITY : m * L.scale + __logf(l);
          __syncwarp();
          unsigned int bad = __ballot_sync(0xffffffffu, row < L.T && test != 0.f);
          while (bad) {
            const int src = __ffs(bad) - 1;
            bad &= bad - 1;
            const int i = row - lane + src;
            put_row(stage, r - lane + src,
                    out_row(L, h, i, __shfl_sync(0xffffffffu, row_begin, src)), DP / 64);
          }
          ptx::fence_proxy_async_smem();
          if (t == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
          else asm volatile("bar.sync 2, 128;" ::: "memory");
          if (r == 0) {
#pragma unroll
            for (int i = 0; i < DP / 64; ++i)
              ptx::tma_store_3d(&M.out, 64 * i, h, row0 + 128 * t, stage + i * kSlab);
            ptx::bulk_commit();
            ptx::bulk_wait<0>();
          }
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
cudaError_t launch(const AttentionMaps& m, const AttentionLaunch& l, cudaStream_t s) {
  static_assert(Cfg<DP>::kSmem <= 232448, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(attention_fwd_kernel<DP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<DP>::kSmem);
  if (e != cudaSuccess) return e;
  const int pairs = (l.T + 128 * kTiles - 1) / (128 * kTiles);
  attention_fwd_kernel<DP><<<pairs * l.hq, kThreads, Cfg<DP>::kSmem, s>>>(m, l);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const AttentionMaps& m, const AttentionLaunch& l, cudaStream_t s) {
  return l.dim <= 64 ? launch<64>(m, l, s) : launch<128>(m, l, s);
}

}  // namespace muon
