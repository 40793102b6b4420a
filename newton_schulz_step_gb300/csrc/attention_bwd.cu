// attention_bwd.cu -- gradients of causal attention over packed sequences with grouped
// key/value heads, on the tensor cores.
//
// With p_ij = exp(scale q_i . k_j - lse_i) and delta_i = dout_i . out_i,
//   ds_ij = p_ij (dout_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i.
// Two kernels, each of which holds its sums in TMEM from the first block to the last:
// one owns 128 queries and walks their keys (dq), one owns 128 keys and walks their
// queries, over all query heads of the group (dk, dv).  S and dP are computed in both:
// seven products a block instead of five.  In return nothing is added in global memory:
// no fp32 dq buffer of 2 x (4 + 4) bytes an element and key block to move, no atomics,
// the same bits in every run.
// p and ds are rounded to bf16, the tensor cores' input; everything else is fp32.  What
// these roundings (2^-9 on average) may add up to, next to the result's own:
//   dv: p rounded -- 1.4 times the result's own rounding error
//   dk: ds rounded, 1.4 times.  delta is not taken from the bf16 out here (that would make
//       it 1.6): sum_j p_ij (dp_ij - delta_i) = 0 at the exact delta, so the row sums that
//       the dq kernel ends with correct it
//   dq: ds rounded, and delta from the bf16 out: 1.6 times; with the remainders of ds of
//       half the columns in a second bf16, 1.4 times.
// Rows that see few keys have few roundings to average, and p near 1 times the error of
// delta: 2 to 3 times on sequences of 2 to 20 tokens.  Those rows' keys are mostly in the
// row's own block.  There, where a sequence begins in the tile, the dq kernel takes delta
// from the block itself (sum ds = 0), and all remainders: 1.0 times.  The dk kernel takes
// the remainders of the block where a sequence ends in the tile: its sums over few queries
// scatter up to 1.7 times without them.  That is a block of a walk in both cases: 8192
// packed tokens, 16/4 heads of 128, dq 142 to 144 us, dk/dv 168 either way.
//
// Warps 0-15 compute, warp 16 issues the copies, warp 17 the products.  A compute thread
// owns a row (TMEM lane) of S and dP and 32 of its columns; each of the 4 groups of warps
// writes P and dS over half of its own columns of S or dP, as bf16 pairs, from where they
// are the A operand of the accumulating product.
#include "attention.cuh"

#include <type_traits>

namespace muon {
namespace {

using namespace attn;

// 16 compute warps in 4 groups, a warp for the copies, a warp for the products: with four
// compute warps on each of the SM's four schedulers a thread has 96 registers, and a warp's
// waits, exponentials and TMEM accesses run beside the others'.  (8 warps with 64 columns
// a thread: dk/dv of 8192 tokens, 32/8 heads of 128, in 751 us instead of 663.)
constexpr int kThreads = 576;
constexpr int kProducerWarp = 16, kMmaWarp = 17;
constexpr uint32_t kStatBytes = 1024;      // a block's 128 log-sum-exps and 128 deltas

__device__ __forceinline__ void compute_barrier() {   // the 16 compute warps
  asm volatile("bar.sync 1, 512;" ::: "memory");
}
__device__ __forceinline__ void half_barrier(int half) {   // the lower or upper 8 of them
  asm volatile("bar.sync %0, 256;" ::"r"(2 + half) : "memory");
}

// ------------------------------------------------------------------ dq
// TMEM: S (0, with heads of 64 or less two buffers: 0 and 320), dP (128; dS over it), dq
// (256), Q and dO (from 512 - DP) as bf16 pairs.  The first block's S and dP take Q and dO
// from where the copies left them; meanwhile the compute warps put both in TMEM for the
// other blocks, whose products then read half as much shared memory (with Q and dO from
// there a step ran 106 cycles instead of 64).
// Per block, in the tensor cores' order, one buffer of S: S of the next block (once the
// exponentials have read this one), dq += dS K, dP of the next block; two buffers: dq,
// dP of the next block, S of the one after.
// What bounds it: heads of 128, the chain dP -> dS -> dq -> dP of the next block: dS is
// written over dP, TMEM has no room for a second one.  8192 tokens, 32/8 heads: 670 us, its
// products at 77 % of a library product's rate (tensor cores active 61 % of the cycles).
// (Handing over dS before its remainders: 1 % less.  Blocks of 64 keys: 815.)
template <int DP> struct DqCfg {
  static constexpr uint32_t kTile = DP / 64 * kSlab;
  static constexpr int kK = DP == 128 ? 3 : 4, kV = DP == 128 ? 2 : 4;   // ring slots
  static constexpr uint32_t kDo = kTile, kKRing = 2 * kTile, kVRing = kKRing + kK * kTile;
  static constexpr uint32_t kMisc = kVRing + kV * kTile, kMiscBytes = 2560;
  static constexpr uint32_t kSmem = kMisc + kMiscBytes;
  static constexpr bool kTwoS = DP == 64;
  static constexpr uint32_t kQCol = 512 - DP, kDoCol = kQCol + DP / 2;
  static __device__ __forceinline__ uint32_t s_col(int j) { return kTwoS && (j & 1) ? 320 : 0; }
};

struct DqMisc {
  uint64_t q_full, q_ready, k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], s_read, dp_full, ds_full, dq_full, drain;
  uint32_t tmem;
  int bad, skip;
  int first, last;                 // begin of the tile's first and last row
  int starts;                      // a sequence begins in the tile
  unsigned int repair[4];          // rows to compute again, by warp of the tile
  float delta[4][128];             // parts of delta
};
static_assert(sizeof(DqMisc) <= DqCfg<64>::kMiscBytes, "misc block");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dq_kernel(const __grid_constant__ AttentionMaps M,
                        const __grid_constant__ AttentionLaunch L) {
  using C = DqCfg<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  DqMisc& X = *reinterpret_cast<DqMisc*>(sm + C::kMisc);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (warp == kProducerWarp && lane == 0) {
    ptx::mbar_init(&X.q_full, 2);
    ptx::mbar_init(&X.q_ready, 16);
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(&X.k_full[s], 1);
      ptx::mbar_init(&X.k_empty[s], 1);
      ptx::mbar_init(&X.v_full[s], 1);
      ptx::mbar_init(&X.v_empty[s], 1);
    }
    ptx::mbar_init(&X.s_full[0], 1);
    ptx::mbar_init(&X.s_full[1], 1);
    ptx::mbar_init(&X.s_read, 16);
    ptx::mbar_init(&X.dp_full, 1);
    ptx::mbar_init(&X.ds_full, 16);
    ptx::mbar_init(&X.dq_full, 1);
    ptx::mbar_init(&X.drain, 1);
    X.bad = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&M.q);
    ptx::prefetch_tmap(&M.dout);
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
  const int tiles = (L.T + 127) / 128;
  const int h = static_cast<int>(blockIdx.x) % L.hq;
  const int tile = tiles - 1 - static_cast<int>(blockIdx.x) / L.hq;
  const int row0 = 128 * tile, kh = h / L.group;

  if (tid < 2) {
    const int b = sequence_of(L, tid ? min(row0 + 127, L.T - 1) : row0).begin;
    if (tid) X.last = b;
    else X.first = b;
  }
  if (tid == 2) {
    const int used = tokens_in_use(L);
    X.starts = row0 < used && sequence_of(L, min(row0 + 127, used - 1)).begin >= row0;
  }
  if (tid < 4) X.repair[tid] = 0;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const Guard guard{&X.bad, L.status,
                    warp == kProducerWarp ? kErrTimeoutProducer
                    : warp == kMmaWarp    ? kErrTimeoutMma
                                          : kErrTimeoutEpilogue};
  const bool run = !X.skip;
  const int begin = __shfl_sync(0xffffffffu, X.first, 0) / kBlock;
  const int n = tile + 1 - begin;                               // key blocks

  if (warp >= kProducerWarp) {
    if (run && warp == kProducerWarp) {
      if (lane == 0) {
        load_tile<DP>(sm, &M.q, h, row0, &X.q_full);
        load_tile<DP>(sm + C::kDo, &M.dout, h, row0, &X.q_full);
        int j = 0;
        bool ok = true;
        for (; j < n && ok; ++j) {
          const int ks = j % C::kK, vs = j % C::kV, row = (begin + j) * kBlock;
          if (j >= C::kK) ok = guard.wait_or_fail(&X.k_empty[ks], (j / C::kK - 1) & 1);
          if (!ok) break;
          load_tile<DP>(sm + C::kKRing + ks * C::kTile, &M.k, kh, row, &X.k_full[ks]);
          if (j >= C::kV) ok = guard.wait_or_fail(&X.v_empty[vs], (j / C::kV - 1) & 1);
          if (!ok) break;
          load_tile<DP>(sm + C::kVRing + vs * C::kTile, &M.v, kh, row, &X.v_full[vs]);
        }
        if (!ok) {                       // copies in flight land before the CTA ends
          ptx::mbar_wait(&X.q_full, 0, nullptr, nullptr, kDrainNs);
          for (int i = j > C::kK ? j - C::kK : 0; i <= j; ++i) {
            ptx::mbar_wait(&X.k_full[i % C::kK], (i / C::kK) & 1, nullptr, nullptr, kDrainNs);
            if (i < j)
              ptx::mbar_wait(&X.v_full[i % C::kV], (i / C::kV) & 1, nullptr, nullptr, kDrainNs);
          }
        }
      }
    } else if (run && warp == kMmaWarp) {
      const uint32_t base = tile_address(sm);
      Ring<C::kK> at_s, at_q;            // K tiles as read by S and by dq
      Ring<C::kV> at_v;
      const int starts = __shfl_sync(0xffffffffu, X.starts, 0);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && guard.issue_wait(bar, parity);
        if (ok) ptx::tc_fence_after();
        return ok;
      };
      // Waits for copies stand where nothing depends on them yet, and products that follow
      // one another go out together: every step of this warp between them costs the
      // tensor cores 100 cycles and more.  (A commit waits for all products before it: the
      // one that frees a tile comes right behind the product that reads it last.)
      auto scores = [&](int j) {           // (the K tile has landed)
        const uint32_t k = base + C::kKRing + at_s.slot * C::kTile;
        if (j == 0) mma_heads<DP>(0, base, k);
        else mma_heads_ts<DP>(C::s_col(j), C::kQCol, k);
        ptx::mma_commit(&X.s_full[C::kTwoS ? j & 1 : 0]);
      };
      auto dp = [&](int j) {               // (the V tile has landed)
        const uint32_t v = base + C::kVRing + at_v.slot * C::kTile;
        if (j == 0) mma_heads<DP>(128, base + C::kDo, v);
        else mma_heads_ts<DP>(128, C::kDoCol, v);
        ptx::mma_commit(&X.dp_full);
        ptx::mma_commit(&X.v_empty[at_v.slot]);
      };
      auto k_landed = [&] { return wait(&X.k_full[at_s.slot], at_s.parity); };
      auto v_landed = [&] { return wait(&X.v_full[at_v.slot], at_v.parity); };
      if (wait(&X.q_full, 0) && k_landed() && v_landed() && ptx::elect_one()) {
        scores(0);
        dp(0);
      }
      at_s.next();
      at_v.next();
      if (n > 1) wait(&X.q_ready, 0);
      if (C::kTwoS && n > 1) {
        if (k_landed() && ptx::elect_one()) scores(1);
        at_s.next();
      }
      for (int j = 0; j < n && ok; ++j) {
        if (!C::kTwoS && j + 1 < n) {
          if (k_landed() && wait(&X.s_read, j & 1) && ptx::elect_one()) scores(j + 1);
          at_s.next();
        }
        if (C::kTwoS && j + 2 < n) k_landed();
        if (j + 1 < n) v_landed();
        if (!ok || !wait(&X.ds_full, j & 1)) break;
        if (ptx::elect_one()) {
          const uint32_t k = base + C::kKRing + at_q.slot * C::kTile;
          mma_rows<DP, 128, 16>(256, 128, k, j > 0);
          if (starts && j + 1 == n) {    // the remainders
            mma_rows<DP, 128, 16>(256, 128 + 16, k, true);
          } else {                       // of keys 0-15 of each group's 32
            constexpr uint32_t kId = ptx::idesc_bf16(128, DP, true);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              ptx::mma_bf16_ts(256, 128 + 32 * i + 16, desc_mn(k, 2 * i), kId, 1);
          }
          ptx::mma_commit(&X.k_empty[at_q.slot]);
          if (j + 1 == n) ptx::mma_commit(&X.dq_full);
          if (j + 1 < n) dp(j + 1);
          if (C::kTwoS && j + 2 < n) scores(j + 2);
        }
        __syncwarp();
        at_q.next();
        at_v.next();
        if (C::kTwoS) at_s.next();
      }
      if (!ok) {                         // products in flight end before TMEM is freed
        if (ptx::elect_one()) ptx::mma_commit(&X.drain);
        ptx::mbar_wait(&X.drain, 0, nullptr, nullptr, kDrainNs);
        __syncwarp();
      }
    }
  } else if (run) {
    const int group = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane, row = row0 + r;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const int used = tokens_in_use(L);
    const int row_begin = row < L.T ? sequence_of(L, row).begin : row + 1;
    const int last_begin = X.last, starts = X.starts;
    const float c = L.scale * kLog2e;
    // delta, 32 columns of a row each; lse in base 2, +inf (p = 0) for rows without keys
    float delta = 0.f, lse2 = INFINITY;
    uint4 o[4];
    const bool columns = 32 * group < DP;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_uint4(0, 0, 0, 0);
    if (row < used) {
      const __nv_bfloat16* out = L.o.row(row, h) + 32 * group;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (columns && 32 * group + 8 * i < L.dim)
          o[i] = *reinterpret_cast<const uint4*>(out + 8 * i);
      lse2 = L.lse[static_cast<size_t>(h) * L.T + row] * kLog2e;
    }
    bool ok = guard.warp_wait(&X.q_full, 0);
    if (ok && columns) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 g = *reinterpret_cast<const uint4*>(sm + C::kDo + tile_off(r, 4 * group + i));
        w[4 * i] = g.x; w[4 * i + 1] = g.y; w[4 * i + 2] = g.z; w[4 * i + 3] = g.w;
        const uint32_t u[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          delta = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(w[4 * i + e] << 16), delta);
          delta = fmaf(__uint_as_float(u[e] & 0xffff0000u),
                       __uint_as_float(w[4 * i + e] & 0xffff0000u), delta);
        }
      }
      ptx::tmem_st16(lanes + C::kDoCol + 16 * group, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(sm + tile_off(r, 4 * group + i));
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
      ptx::tmem_st16(lanes + C::kQCol + 16 * group, w);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&X.q_ready);
    X.delta[group][r] = row < used ? delta : 0.f;
    compute_barrier();
    delta = (X.delta[0][r] + X.delta[1][r]) + (X.delta[2][r] + X.delta[3][r]);
    float* const stats = L.stats + (static_cast<size_t>(h) * tiles + tile) * 256 + r;
    if (group == 0) stats[0] = lse2;
    const uint64_t c2 = pair(c, c), lse22 = pair(-lse2, -lse2), delta2 = pair(-delta, -delta);
    uint64_t rest = 0;                                 // of the row's sum of ds
    auto step = [&](int j, auto own) {                 // own: the rows' own block, with starts
      const int k0 = (begin + j) * kBlock;
      ok = C::kTwoS ? guard.warp_wait(&X.s_full[j & 1], (j >> 1) & 1)
                    : guard.warp_wait(&X.s_full[0], j & 1);
      if (!ok) return;
      ptx::tc_fence_after();
      uint32_t x[32];
      uint64_t p[16];
      ptx::tmem_ld32_sync(lanes + C::s_col(j) + 32 * group, x);
      if (!C::kTwoS) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&X.s_read);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 y = unpair(
            fma2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, lse22));
        p[i] = pair(ex2(y.x), ex2(y.y));
      }
      ok = guard.warp_wait(&X.dp_full, j & 1);
      if (!ok) return;
      ptx::tc_fence_after();
      ptx::tmem_ld32_sync(lanes + 128 + 32 * group, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 y = unpair(mul2(
            p[i], add2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), delta2)));
        x[2 * i] = __float_as_uint(y.x);
        x[2 * i + 1] = __float_as_uint(y.y);
      }
      bool clear = false;
      if (k0 < last_begin || j + 1 == n) {
        clear = k0 < X.first || used < min(k0 + kBlock, L.T);
        hide(x, row_begin - k0 - 32 * group, row - k0 - 32 * group, 0u);
      }
      if constexpr (decltype(own)::value) {
        // rows that see keys of this block only: their delta is the one of sum ds = 0
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) part += __uint_as_float(x[i]);
        compute_barrier();                             // (delta's parts have been read)
        X.delta[group][r] = row_begin >= k0 ? part : 0.f;
        compute_barrier();
        const float e = (X.delta[0][r] + X.delta[1][r]) + (X.delta[2][r] + X.delta[3][r]);
        delta += e;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = unpair(fma2(
              p[i], pair(-e, -e), pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]))));
          x[2 * i] = __float_as_uint(y.x);
          x[2 * i + 1] = __float_as_uint(y.y);
        }
        hide(x, row_begin - k0 - 32 * group, row - k0 - 32 * group, 0u);
        uint32_t remainder[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = __uint_as_float(x[16 + 2 * i]), b = __uint_as_float(x[17 + 2 * i]);
          const uint32_t w = pack2(a, b);
          remainder[i] =
              pack2(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xffff0000u));
        }
        ptx::tmem_st8(lanes + 128 + 32 * group + 24, remainder);
      }
      uint32_t w[16], remainder[8];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = __uint_as_float(x[2 * i]), b = __uint_as_float(x[2 * i + 1]);
        w[i] = pack2(a, b);
        rest = add2(rest, pair(a, b));
        if (i < 8)
          remainder[i] = pack2(a - __uint_as_float(w[i] << 16),
                               b - __uint_as_float(w[i] & 0xffff0000u));
      }
      ptx::tmem_st16(lanes + 128 + 32 * group, w);
      ptx::tmem_st8(lanes + 128 + 32 * group + 16, remainder);
      if (clear) {                       // the block holds padding, or keys before those that
        const int s = j % C::kK;         // the tile sees: clear them (S has read the tile)
        if (group == 0 && (k0 + r < X.first || k0 + r >= used))
          zero_row<DP>(sm + C::kKRing + s * C::kTile, r);
        ptx::fence_proxy_async_smem();
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&X.ds_full);
    };
    for (int j = 0; j + starts < n && ok; ++j) step(j, std::false_type{});
    if (starts && ok) step(n - 1, std::true_type{});
    if (starts && !ok) {        // a wait ran out: others may stand at that step's two barriers
      compute_barrier();
      compute_barrier();
    }
    if (ok) ok = guard.warp_wait(&X.dq_full, 0);
    if (ok && 32 * group < DP) {
      ptx::tc_fence_after();
      // Q has been read for the last time: dq goes through its place
      float test = 0.f;                                // NaN if an element is not finite
      uint32_t o[32];
      ptx::tmem_ld32_sync(lanes + 256 + 32 * group, o);
      float f[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        f[e] = row < used ? __uint_as_float(o[e]) * L.scale : 0.f;     // (no gradient of padding)
        test = fmaf(f[e], 0.f, test);
      }
      store_row32(sm, r, 4 * group, f);
      const unsigned int bad = __ballot_sync(0xffffffffu, test != 0.f);
      if (bad && lane == 0) atomicOr(&X.repair[quarter], bad);
    }
    if (ok) {
      const float2 a = unpair(rest);
      X.delta[group][r] = a.x + a.y;
    }
    compute_barrier();                                 // (reached by every compute thread)
    if (ok) {
      if (group == 1)                // (0 of rows that are not there: where nothing is hidden, a
        stats[128] =                 // value that is not finite reaches their ds)
            row < used
                ? delta + ((X.delta[0][r] + X.delta[1][r]) + (X.delta[2][r] + X.delta[3][r]))
                : 0.f;
      // Any part of a row may be bad: the four warps of the rows share the joint set.  (A row
      // whose visible ds, summed up here, are not finite is so throughout.)
      unsigned int bad = X.repair[quarter];
      if (bad) {
        const float sum = (X.delta[0][r] + X.delta[1][r]) + (X.delta[2][r] + X.delta[3][r]);
        bad &= __ballot_sync(0xffffffffu, isfinite(sum)) & (0x11111111u << group);
        mend_dq(L, sm, DP / 64, h, row0, r - lane, row_begin, bad);
      }
      ptx::fence_proxy_async_smem();
    }
    compute_barrier();
    if (ok && tid == 0 && !X.bad) {
#pragma unroll
      for (int i = 0; i < DP / 64; ++i)
        ptx::tma_store_3d(&M.dq, 64 * i, h, row0, sm + i * kSlab);
      ptx::bulk_commit();
      ptx::bulk_wait_read<0>();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(X.tmem, 512);
  }
}

// ------------------------------------------------------------------ dk, dv
// Scores are transposed here (rows are keys): P^T and dS^T are A operands as they come,
// without an exchange.  TMEM: S^T (0; with heads of 64 or less a second buffer: 384),
// dP^T (128), dv (256), dk (256 + DP).  Per block, in the tensor cores' order:
// dv += P^T dO, S^T of the next block (two buffers: of the one after), dk += dS^T Q, dP^T
// of the next block; so P of a block is computed beside the last two products of the one
// before, and dS beside the first two of its own.  With heads of 128 the four products
// bound it: 87 % of the rate that a library product reaches (8192 tokens, 32/8 heads: 672
// us).  With 64 the exponentials do, and the second buffer keeps the compute warps from
// waiting for S.
// Where the tiles leave SMs without work, 2 or 4 blocks of a cluster share a tile: each
// walks its part of the queries, and they add up each other's sums through distributed
// shared memory, in the order of their ranks.
template <int DP> struct DkvCfg {
  static constexpr uint32_t kTile = DP / 64 * kSlab;
  static constexpr int kStages = DP == 128 ? 2 : 4;          // of Q (with its stats) and dO
  static constexpr uint32_t kV = kTile, kQRing = 2 * kTile, kDoRing = kQRing + kStages * kTile;
  static constexpr uint32_t kStats = kDoRing + kStages * kTile;
  static constexpr uint32_t kMisc = kStats + kStages * kStatBytes;
  static constexpr uint32_t kSmem = kMisc + 1024;
  static constexpr bool kTwoS = DP == 64;
  static constexpr int kAhead = kTwoS ? 2 : 1;   // S of which block follows dv of one
  static __device__ __forceinline__ uint32_t s_col(int i) { return kTwoS && (i & 1) ? 384 : 0; }
};

struct DkvMisc {
  uint64_t kv_full, q_full[4], q_empty[4], do_full[4], do_empty[4];
  uint64_t s_full[2], dp_full, p_full[2], ds_full, done, drain;
  uint32_t tmem;
  int bad, skip;
  int used;                        // tokens that belong to a sequence
  int first_end, blocks;           // end of the first key's sequence; query blocks per head
  int key_end[kBlock];             // end of each key's sequence (no register is left for it)
  int lost;                        // dout has been cleared where keys see it
};
static_assert(sizeof(DkvMisc) <= 1024, "misc block");

// Byte offset of 4 sums (columns 4 c .. 4 c + 3 of row r of dv or dk): rows of DP fp32 in
// the place of the Q and dO rings, 16-byte columns permuted so that neither a warp's 32
// rows nor its 32 columns meet in a bank.
template <int DP>
__device__ __forceinline__ uint32_t sum_off(int which, int r, int c) {
  static_assert(2u * 128u * DP * 4u <= DkvCfg<DP>::kStats - DkvCfg<DP>::kQRing, "room for the sums");
  return DkvCfg<DP>::kQRing + ((which * 128 + r) * (DP / 4) + (c ^ (r & (DP / 4 - 1)))) * 16;
}

// Clears what is not finite in row r of a tile of Q or dO; whether there was any.
template <int DP>
static __device__ __noinline__ bool clear_row(uint8_t* tile, int r) {
  bool any = false;
  for (int c = 0; c < DP / 2; ++c) {
    uint32_t* p = reinterpret_cast<uint32_t*>(tile + tile_off(r, c >> 2)) + (c & 3);
    uint32_t w = *p;
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    if (w == *p) continue;
    *p = w;
    any = true;
  }
  return any;
}

// Puts NaN into dv where a dout that is not finite belongs and has been cleared: rows r0, r0 + 2,
// ... r0 + 30, staged as bf16 (`stage`) or as sums.
template <int DP>
static __device__ __noinline__ void mark_lost(const AttentionLaunch& L, uint8_t* sm, uint8_t* stage,
                                              int kh, int key0, int r0, const int* key_end) {
  Behind behind;
  for (int r = r0; r < r0 + 32; r += 2) {
    if (key_end[r] <= key0 + r) continue;                  // no key of a sequence
    const unsigned int lost = lost_columns(L, kh, key0, key0 + r, key_end[r], behind);
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) {
      if (!(lost >> e & 1u)) continue;
      const int col = 64 * (e >> 1) + 2 * static_cast<int>(threadIdx.x & 31) + (e & 1);
      if (stage)
        *reinterpret_cast<uint16_t*>(stage + tile_off(r, col >> 3) + 2 * (col & 7)) = 0x7fff;
      else
        *reinterpret_cast<float*>(sm + sum_off<DP>(0, r, col >> 2) + 4 * (col & 3)) = NAN;
    }
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dkv_kernel(const __grid_constant__ AttentionMaps M,
                         const __grid_constant__ AttentionLaunch L) {
  using C = DkvCfg<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  DkvMisc& X = *reinterpret_cast<DkvMisc*>(sm + C::kMisc);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (warp == kProducerWarp && lane == 0) {
    ptx::mbar_init(&X.kv_full, 2);
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(&X.q_full[s], 1);
      ptx::mbar_init(&X.q_empty[s], 1);
      ptx::mbar_init(&X.do_full[s], 1);
      ptx::mbar_init(&X.do_empty[s], 1);
    }
    ptx::mbar_init(&X.s_full[0], 1);
    ptx::mbar_init(&X.s_full[1], 1);
    ptx::mbar_init(&X.dp_full, 1);
    ptx::mbar_init(&X.p_full[0], 16);
    ptx::mbar_init(&X.p_full[1], 16);
    ptx::mbar_init(&X.ds_full, 16);
    ptx::mbar_init(&X.done, 1);
    ptx::mbar_init(&X.drain, 1);
    X.bad = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&M.q);
    ptx::prefetch_tmap(&M.dout);
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

  // of one sequence, the first tiles are seen by the most queries: they go first
  const int tiles = (L.T + 127) / 128;
  const int rank = L.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int kh = static_cast<int>(blockIdx.x) / L.split % L.hk;
  int tile = static_cast<int>(blockIdx.x) / L.split / L.hk;
  if (L.ranked)
    tile = ranked_tile(tiles, tile, reinterpret_cast<int*>(sm), [&](int i) {
      const Span s = sequence_of(L, min(128 * i + 127, L.T - 1));
      return s.end / kBlock - i;
    });
  const int key0 = 128 * tile;

  if (tid == 0) {
    const int used = tokens_in_use(L);
    int end = 0;
    if (key0 < used) end = sequence_of(L, min(key0 + 127, used - 1)).end;
    X.used = used;
    X.lost = 0;
    X.first_end = sequence_of(L, key0).end;
    X.blocks = end > key0 ? (end - 1) / kBlock + 1 - tile : 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const Guard guard{&X.bad, L.status,
                    warp == kProducerWarp ? kErrTimeoutProducer
                    : warp == kMmaWarp    ? kErrTimeoutMma
                                          : kErrTimeoutEpilogue};
  const bool run = !X.skip;
  const int blocks = __shfl_sync(0xffffffffu, X.blocks, 0);
  // query blocks of all heads, and this block's part of them
  const int all = blocks * L.group;
  const int first = all * rank / L.split, n = all * (rank + 1) / L.split - first;

  if (warp >= kProducerWarp) {
    if (run && n > 0 && warp == kProducerWarp) {
      if (lane == 0) {
        load_tile<DP>(sm, &M.k, kh, key0, &X.kv_full);
        load_tile<DP>(sm + C::kV, &M.v, kh, key0, &X.kv_full);
        int i = 0, h = kh * L.group + first / blocks, b = tile + first % blocks;
        bool ok = true;
        for (; i < n; ++i) {
          const int s = i % C::kStages;
          if (i >= C::kStages) ok = guard.wait_or_fail(&X.q_empty[s], (i / C::kStages - 1) & 1);
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(&X.q_full[s], C::kTile + kStatBytes);
#pragma unroll
          for (int e = 0; e < DP / 64; ++e)
            ptx::tma_load_3d(sm + C::kQRing + s * C::kTile + e * kSlab, &M.q, 64 * e, h,
                             b * kBlock, &X.q_full[s]);
          ptx::bulk_load(sm + C::kStats + s * kStatBytes,
                         L.stats + (static_cast<size_t>(h) * tiles + b) * 256, kStatBytes,
                         &X.q_full[s]);
          if (i >= C::kStages) ok = guard.wait_or_fail(&X.do_empty[s], (i / C::kStages - 1) & 1);
          if (!ok) break;
          load_tile<DP>(sm + C::kDoRing + s * C::kTile, &M.dout, h, b * kBlock, &X.do_full[s]);
          if (++b == tile + blocks) {
            b = tile;
            ++h;
          }
        }
        if (!ok) {                       // copies in flight land before the CTA ends
          ptx::mbar_wait(&X.kv_full, 0, nullptr, nullptr, kDrainNs);
          for (int e = i > C::kStages ? i - C::kStages : 0; e <= i; ++e) {
            const uint32_t parity = (e / C::kStages) & 1;
            ptx::mbar_wait(&X.q_full[e % C::kStages], parity, nullptr, nullptr, kDrainNs);
            if (e < i)
              ptx::mbar_wait(&X.do_full[e % C::kStages], parity, nullptr, nullptr, kDrainNs);
          }
        }
      }
    } else if (run && n > 0 && warp == kMmaWarp) {
      const uint32_t base = tile_address(sm);
      Ring<C::kStages> at_s, at_p, at_v, at_k;   // tiles as read by S, dP, dv and dk
      const int ends = __shfl_sync(0xffffffffu, X.first_end, 0) <= key0 + kBlock;
      int b = first % blocks;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && guard.issue_wait(bar, parity);
        if (ok) ptx::tc_fence_after();
        return ok;
      };
      // (With 4 tiles in a ring the waits for copies stand early, as in the dq kernel; with 2
      // the next tile may land late, and what does not need it goes first: 784 us with early
      // waits, 670 with late ones, for 8192 tokens, 32/8 heads of 128.)
      constexpr bool kEarly = C::kStages > 2;
      auto scores = [&](int i) {           // (the Q tile has landed)
        mma_heads<DP>(C::s_col(i), base, base + C::kQRing + at_s.slot * C::kTile);
        ptx::mma_commit(&X.s_full[C::kTwoS ? i & 1 : 0]);
      };
      auto dp = [&] {                      // (the dO tile has landed)
        mma_heads<DP>(128, base + C::kV, base + C::kDoRing + at_p.slot * C::kTile);
        ptx::mma_commit(&X.dp_full);
      };
      auto q_landed = [&] { return wait(&X.q_full[at_s.slot], at_s.parity); };
      auto do_landed = [&] { return wait(&X.do_full[at_p.slot], at_p.parity); };
      if (wait(&X.kv_full, 0) && q_landed() && ptx::elect_one()) scores(0);
      at_s.next();
      if (ok && do_landed() && ptx::elect_one()) dp();
      at_p.next();
      if (C::kTwoS && n > 1) {
        if (ok && q_landed() && ptx::elect_one()) scores(1);
        at_s.next();
      }
      for (int i = 0; i < n && ok; ++i) {
        if (kEarly && i + C::kAhead < n) q_landed();
        if (!ok ||
            !(C::kTwoS ? wait(&X.p_full[i & 1], (i >> 1) & 1) : wait(&X.p_full[0], i & 1)))
          break;
        if (ptx::elect_one()) {
          mma_rows<DP, 128, 16>(256, C::s_col(i), base + C::kDoRing + at_v.slot * C::kTile, i > 0);
          ptx::mma_commit(&X.do_empty[at_v.slot]);
          if (kEarly && i + C::kAhead < n) scores(i + C::kAhead);
        }
        __syncwarp();
        if (!kEarly && i + C::kAhead < n && q_landed() && ptx::elect_one()) scores(i + C::kAhead);
        at_v.next();
        at_s.next();
        if (kEarly && i + 1 < n) do_landed();
        if (!ok || !wait(&X.ds_full, i & 1)) break;
        if (ptx::elect_one()) {
          const uint32_t q = base + C::kQRing + at_k.slot * C::kTile;
          mma_rows<DP, 128, 16>(256 + DP, 128, q, i > 0);
          if (ends && b == 0) mma_rows<DP, 128, 16>(256 + DP, 128 + 16, q, true);
          ptx::mma_commit(&X.q_empty[at_k.slot]);
          if (i + 1 == n) ptx::mma_commit(&X.done);
          if (kEarly && i + 1 < n) dp();
        }
        __syncwarp();
        if (!kEarly && i + 1 < n && do_landed() && ptx::elect_one()) dp();
        at_k.next();
        at_p.next();
        if (++b == blocks) b = 0;
      }
      if (!ok) {                         // products in flight end before TMEM is freed
        if (ptx::elect_one()) ptx::mma_commit(&X.drain);
        ptx::mbar_wait(&X.drain, 0, nullptr, nullptr, kDrainNs);
        __syncwarp();
      }
    }
  } else if (run) {
    const int group = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane, key = key0 + r;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    if (group == 0) X.key_end[r] = key < X.used ? sequence_of(L, key).end : key;
    compute_barrier();
    const int first_end = X.first_end;
    const float c = L.scale * kLog2e;
    const uint64_t c2 = pair(c, c);
    bool ok = true;
    int b = n > 0 ? tile + first % blocks : tile;
    Ring<C::kStages> at;
    auto step = [&](int i, auto own) {                 // own: the keys' own block, with ends
      const int q0 = b * kBlock;
      const bool masked = b == tile || q0 + kBlock > first_end;
      auto hide_unseen = [&](uint32_t (&s)[32]) {
        hide(s, key - q0 - 32 * group, X.key_end[r] - 1 - q0 - 32 * group, 0u);
      };
      const float4* lse2 =
          reinterpret_cast<const float4*>(sm + C::kStats + at.slot * kStatBytes) + 8 * group;
      ok = guard.warp_wait(&X.q_full[at.slot], at.parity);            // the stats
      if (!ok) return;
      // Where a key may not see a query, what is not finite in its q and dout would reach the key
      // all the same.  A query that holds any, or that is padding, has a log-sum-exp or a delta
      // that is not finite; its own keys have NaN for p or for ds then.
      unsigned int gone = 0;                           // such queries of this warp's columns
      if (masked) {
        const float* z = reinterpret_cast<const float*>(lse2) + lane;
        gone = __ballot_sync(0xffffffffu, q0 + 32 * group + lane < L.T &&
                                              !(fabsf(z[0]) + fabsf(z[128]) < INFINITY));
      }
      ok = (C::kTwoS ? guard.warp_wait(&X.s_full[i & 1], (i >> 1) & 1)
                     : guard.warp_wait(&X.s_full[0], i & 1));
      if (!ok) return;
      ptx::tc_fence_after();
      uint32_t x[32];
      uint64_t p[16];
      const uint32_t ts = lanes + C::s_col(i) + 32 * group, tp = lanes + 128 + 32 * group;
      ptx::tmem_ld32_sync(ts, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 z = lse2[e];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int o = 4 * e + 2 * k;
          const float2 y =
              unpair(fma2(pair(__uint_as_float(x[o]), __uint_as_float(x[o + 1])), c2,
                          k ? pair(-z.z, -z.w) : pair(-z.x, -z.y)));
          x[o] = __float_as_uint(ex2(y.x));
          x[o + 1] = __float_as_uint(ex2(y.y));
        }
      }
      if (masked) hide_unseen(x);
      {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
          p[e] = pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        }
        ptx::tmem_st16(ts, w);
      }
      if (__builtin_expect(gone != 0, 0)) {
        ok = guard.warp_wait(&X.do_full[at.slot], at.parity);
        if (!ok) return;
        if (quarter < 2 && (gone >> lane & 1u) &&
            clear_row<DP>(sm + (quarter ? C::kDoRing : C::kQRing) + at.slot * C::kTile,
                          32 * group + lane) &&
            quarter == 1 && isfinite(reinterpret_cast<const float*>(lse2)[lane]))
          X.lost = 1;                                  // single columns of dv need it
        ptx::fence_proxy_async_smem();
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&X.p_full[C::kTwoS ? i & 1 : 0]);

      ok = guard.warp_wait(&X.dp_full, i & 1);
      if (!ok) return;
      ptx::tc_fence_after();
      ptx::tmem_ld32_sync(tp, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 z = lse2[32 + e];           // delta
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int o = 4 * e + 2 * k;
          const float2 y =
              unpair(mul2(p[2 * e + k], add2(pair(__uint_as_float(x[o]), __uint_as_float(x[o + 1])),
                                             k ? pair(-z.z, -z.w) : pair(-z.x, -z.y))));
          x[o] = __float_as_uint(y.x);
          x[o + 1] = __float_as_uint(y.y);
        }
      }
      // (p is 0 where a query is not seen, and 0 times the finite dp - delta of the others is 0)
      if (__builtin_expect(gone != 0, 0)) hide_unseen(x);
      {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        ptx::tmem_st16(tp, w);
        if constexpr (decltype(own)::value) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack2(__uint_as_float(x[2 * e]) - __uint_as_float(w[e] << 16),
                         __uint_as_float(x[2 * e + 1]) - __uint_as_float(w[e] & 0xffff0000u));
          ptx::tmem_st16(tp + 16, w);
        }
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&X.ds_full);
      at.next();
      if (++b == tile + blocks) b = tile;
    };
    const bool ends = first_end <= key0 + kBlock;
    for (int i = 0; i < n && ok; ++i) {
      if (ends && b == tile) step(i, std::true_type{});
      else step(i, std::false_type{});
    }
    // V and K have been read for the last time: dv goes through V's place (groups 0, 1),
    // dk through K's (groups 2, 3)
    const int which = group >> 1, side = group & 1;
    uint8_t* stage = which ? sm : sm + C::kV;
    if (ok && n > 0) ok = guard.warp_wait(&X.done, 0);
    if (ok && L.split > 1) {
      // the tiles of Q and dO have been read for the last time: the sums go there
      ptx::tc_fence_after();
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        uint32_t o[32];
        ptx::tmem_ld32_sync(lanes + 256 + DP * which + DP / 2 * side + 32 * i, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4 v = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                 __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          if (n == 0) v = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(
              sm + sum_off<DP>(which, r, DP / 8 * side + 8 * i + e)) = v;
        }
      }
    } else if (ok) {
      ptx::tc_fence_after();
      const float f0 = which ? L.scale : 1.f;
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        const int col = DP / 2 * side + 32 * i;
        uint32_t o[32];
        ptx::tmem_ld32_sync(lanes + 256 + DP * which + col, o);
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          f[e] = key < X.used && n > 0 ? __uint_as_float(o[e]) * f0 : 0.f;
        store_row32(stage, r, col / 8, f);
      }
    }
    half_barrier(which);                               // (reached by every compute thread)
    if (ok) {
      if (__builtin_expect(X.lost && !which, 0))       // (the two warps of a row's sides take
        mark_lost<DP>(L, sm, L.split > 1 ? nullptr : stage, kh, key0, r - lane + side,   // every
                      X.key_end);                                                 // other row)
      ptx::fence_proxy_async_smem();
    }
    half_barrier(which);
    if (ok && L.split == 1 && side == 0 && r == 0 && !X.bad) {
#pragma unroll
      for (int i = 0; i < DP / 64; ++i)
        ptx::tma_store_3d(which ? &M.dk : &M.dv, 64 * i, kh, key0, stage + i * kSlab);
      ptx::bulk_commit();
      ptx::bulk_wait_read<0>();
    }
  }
  if (L.split > 1) {
    // (every thread of every block of the cluster comes here, in bounded time)
    ptx::cluster_arrive();
    ptx::cluster_wait();
    if (run && !X.bad && warp < kProducerWarp) {
      // a warp adds up a row, a lane 4 columns of it
      const int used = X.used, rows = kBlock / L.split;
      for (int i = warp; i < 2 * rows; i += kProducerWarp) {
        const int which = i & 1, r = rank * rows + (i >> 1), key = key0 + r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < DP / 4) {
          const uint32_t at = ptx::smem_u32(sm + sum_off<DP>(which, r, lane));
          for (int c = 0; c < L.split; ++c) {
            const float4 x = ptx::ld_cluster_f4(ptx::mapa_shared(at, c));
            v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
          }
        }
        const float f = key >= used ? 0.f : which ? L.scale : 1.f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
        if (key >= used) v = make_float4(0.f, 0.f, 0.f, 0.f);
        __nv_bfloat16* row = (which ? L.dk : L.dv).row(key, kh);
        if (key < L.T && 4 * lane < L.dim)
          *reinterpret_cast<uint2*>(row + 4 * lane) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
      }
    }
    ptx::cluster_arrive();                             // nobody reads this block's sums any more
    ptx::cluster_wait();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(X.tmem, 512);
  }
}

template <typename K>
cudaError_t launch(K kernel, int heads, int split, uint32_t smem, const AttentionMaps& m,
                   AttentionLaunch& l, cudaStream_t s) {
  l.split = split;
  return launch_behind(kernel, (l.T + 127) / 128 * heads * split, kThreads, smem, m, l, s, split);
}
static_assert(DqCfg<128>::kSmem <= 232448 && DkvCfg<128>::kSmem <= 232448, "shared memory");

}  // namespace

cudaError_t launch_attention_dq(const AttentionMaps& m, AttentionLaunch l, cudaStream_t s) {
  return l.dim <= 64 ? launch(attention_dq_kernel<64>, l.hq, 1, DqCfg<64>::kSmem, m, l, s)
                     : launch(attention_dq_kernel<128>, l.hq, 1, DqCfg<128>::kSmem, m, l, s);
}

cudaError_t launch_attention_dkv(const AttentionMaps& m, AttentionLaunch l, int sms,
                                 cudaStream_t s) {
  // 2 or 4 blocks a tile while that takes no second wave: then the longest tile sets the
  // time (in two waves it was no faster: 128 tiles of 4096 tokens, 8/4 heads of 64, 37 us
  // either way; 80 tiles of 2048 tokens, 5 heads of 80, 28 us instead of 24)
  const int units = (l.T + 127) / 128 * l.hk;
  // ... but of one sequence, whose longest walk is known here to be 2 sms / ((tiles + 1) hk)
  // times an SM's share of all walks: 4096 tokens, 8/4 heads of 64, (2.3 times) 74 us unsplit,
  // 51 split; 8192 tokens (1.2 times) 137 and 147.
  const bool uneven = l.n_seqs <= 1 && ((l.T + 127) / 128 + 1) * l.hk * 3 <= sms * 4;
  const int split = units * 4 <= sms ? 4 : units * 2 <= sms || uneven ? 2 : 1;
  l.ranked = split == 1 && l.group > 1 && rank_tiles(l.n_seqs, (l.T + 127) / 128, l.hk, sms);
  return l.dim <= 64 ? launch(attention_dkv_kernel<64>, l.hk, split, DkvCfg<64>::kSmem, m, l, s)
                     : launch(attention_dkv_kernel<128>, l.hk, split, DkvCfg<128>::kSmem, m, l, s);
}

}  // namespace muon
