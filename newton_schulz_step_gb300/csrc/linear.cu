// linear.cu -- products with a weight matrix: y = act(x W^T + b) + r with everything after
// the product in its epilogue, and the gradients
//   dz = dy act'(z),   dx = dz W,   dW = dz^T x,   db = sum over tokens of dz
//
// All three products are D[i][j] = sum_k A[i][k] B[j][k] of bf16 operands with fp32 sums;
// they differ in which operand lies with its contraction along the rows:
//   y:   A = x  (K-major),   B = W (K-major)
//   dx:  A = dz (K-major),   B = W read by columns (MN-major)
//   dW:  A = dz, B = x, both read by columns (MN-major)
// The tensor cores take either by a bit of the descriptors, so nothing is transposed.
//
// linear_gemm_kernel: persistent clusters of two CTAs, each pair on a 256 x kBN tile with
// cta_group::2 products; 320 threads a CTA:
//   warp 0      TMA producer into a ring of 128-byte swizzled stages, 64 deep in k
//   warp 1      TMEM; in the even CTA the tcgen05.mma issuer
//   warps 2..9  epilogue: two warps share the 32 rows of a TMEM quarter, a half of the
//               columns each; blocks of 32 x 64 go out by TMA, the residual comes in by TMA
// The accumulator is double buffered in TMEM: the epilogue of a tile runs beside the
// products of the next.  Eight epilogue warps (the rounds of the Newton-Schulz kernel have
// four) because a tile of a short contraction is over in 4096 clocks (512 deep), and its
// activation takes as long on four.
// Where the tiles are too few for the pairs, the contraction is split: each split leaves its
// fp32 sums in the workspace, and linear_finish_kernel adds them in order and applies the
// epilogue, so the result does not depend on which split came first.  dx and dW go in one
// launch (two problems): neither fills the card by itself where matrices are small.
//
// What bounds it: the tensor cores.  16384 x 4096 x 4096 takes 290 us (1896 TFLOP/s), a
// library product 275; 8192 x 2048 x 8192 151 and 139; 8192 x 11008 x 4096 387 and 382, back to
// back under the power limit 446 and 444; dx and dW of 8192 x 2048 x 8192 293 us, 88 % of the
// tensor pipe's cycles.  (Sizes: tokens, width in, width out.)  The steps on the way, first size:
//   copies issued from a branch on a lane index took 600 clocks a step of 512 clocks of
//   products, whatever the ring's depth (4 to 6 stages), the order of the tiles or the L2
//   hints; issued by an elected lane of a warp in step: 356 -> 308 us;
//   tile indexes by multiplications instead of divisions: 302;
//   the accumulator released without a cluster-scope release, which waits for the stores
//   before it: 2000 clocks a tile, 291, and 16384 x 64 x 4096 40 -> 29 us.
// 6 stages with one staging slot a warp gain 2 % without a residual and were not kept.
//
// One or two tokens, up to four, would leave a 256-row tile almost empty; the products are
// then bound by reading W once, and linear_token_kernel does it on the CUDA cores.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kSlotBytes = 4096;            // one 32 x 64 bf16 block
constexpr int kSlots = 2;                   // per epilogue warp

template <int kBN>
struct Cfg {
  static constexpr int kABytes = kTileM * kTileK * 2;          // this CTA's 128 rows of A
  static constexpr int kBBytes = (kBN / 2) * kTileK * 2;       // its half of the columns' B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = kBN == 256 ? 5 : 6;
  static constexpr int kTmemCols = 2 * kBN;
  static constexpr int kUnits = kBN / 128;                     // 64-column blocks of a warp
  static constexpr int kStagingBytes = kEpiWarps * kSlots * kSlotBytes;
  static constexpr int kSmem = kStages * kStageBytes + kStagingBytes + 512 + 1024;
};
static_assert(Cfg<256>::kSmem <= 232448 && Cfg<128>::kSmem <= 232448, "227 KB a CTA");

// ------------------------------------------------------------ activations
// GELU's tanh form is z / (1 + exp(-2 u)), u = a (z + b z^3).  The exponential is taken as a
// power of two: 2^(z (c + d z^2)) with c = -2 a log2(e), d = b c.
constexpr float kGeluA = 0.7978845608028654f, kGeluB = 0.044715f;
constexpr float kGeluC = -2.f * kGeluA * 1.4426950408889634f, kGeluD = kGeluB * kGeluC;
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float gelu_gate(float z) {
  return reciprocal_approx(1.f + exp2_approx(z * fmaf(kGeluD * z, z, kGeluC)));
}
// (comparisons that a NaN fails lead to arithmetic on it, so it stays one)
__device__ __forceinline__ float relu2(float z) { return z <= 0.f ? 0.f : z * z; }
template <int kN>
__device__ __forceinline__ void activate(float (&z)[kN], int act) {
  if (act == MUON_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < kN; ++i) z[i] = relu2(z[i]);
  } else if (act == MUON_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kN; ++i) z[i] *= gelu_gate(z[i]);
  }
}
// v times the slope at z
template <int kN>
__device__ __forceinline__ void times_slope(float (&v)[kN], const float (&z)[kN], int act) {
  if (act == MUON_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] *= z[i] <= 0.f ? 0.f : 2.f * z[i];
  } else if (act == MUON_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      // beyond +-30 the slope is 1 or 0 to the last bit, and z^3 may overflow
      const float c = z[i] > 30.f ? 30.f : z[i] < -30.f ? -30.f : z[i];
      const float s = gelu_gate(c);
      v[i] *= fmaf(2.f * c * s * (1.f - s), kGeluA * fmaf(3.f * kGeluB * c, c, 1.f), s);
    }
  }
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]),
                    pack_bf2(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf_lo(w.x); v[1] = bf_hi(w.x); v[2] = bf_lo(w.y); v[3] = bf_hi(w.y);
  v[4] = bf_lo(w.z); v[5] = bf_hi(w.z); v[6] = bf_lo(w.w); v[7] = bf_hi(w.w);
}
// 8 consecutive values from column c of a row of n; those past the row are 0.  p is 16-byte
// aligned where the row and c are.
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int c, int n, float (&v)[8]) {
  if (c + 8 <= n) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(row + c)), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? __bfloat162float(row[c + i]) : 0.f;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    *reinterpret_cast<uint4*>(row + c) = pack8(v);
  } else {
    for (int i = 0; i < 8 && c + i < n; ++i) row[c + i] = __float2bfloat16_rn(v[i]);
  }
}

// ------------------------------------------------------------ tiles
struct Item {
  int p, tile, split, pr, tn, kb0, kb1;
};

// Linear item -> problem, split, tile.  All tiles of a split come before the next split.
// Tiles go by bands of kBand pair rows, column by column within a band: the pairs at work
// at one time then share a few row panels of A and column panels of B in L2.
__device__ __forceinline__ Item decode(const LinearLaunch& L, int item) {
  Item it;
  it.p = L.n_prob > 1 && item >= L.prob[1].item_begin ? 1 : 0;
  const LinearProblem& P = L.prob[it.p];
  const int local = item - P.item_begin;
  it.split = P.by_tiles.quotient(local);
  it.tile = local - it.split * (P.tiles_m * P.tiles_n);
  const int band = P.by_band.quotient(it.tile);
  const int w = it.tile - band * kBand * P.tiles_n;
  const bool whole = band < P.last_band;
  it.tn = whole ? w / kBand : P.by_last.quotient(w);
  it.pr = band * kBand + w - it.tn * (whole ? kBand : P.tiles_m - band * kBand);
  const int each = P.k_each, more = P.k_more;
  it.kb0 = it.split * each + min(it.split, more);
  it.kb1 = it.kb0 + each + (it.split < more ? 1 : 0);
  return it;
}

__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2);
}
// Row r of a 32 x 64 block, as TMA wants it (16-byte unit u of row r at unit u ^ (r & 7)).
__device__ __forceinline__ void stage_row(uint8_t* blk, int r, const float (&v)[64]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(blk + sw128(r, 8 * q)) = pack8(v + 8 * q);
}

// Arrive on the even CTA's barrier, with no memory of this thread to publish: what it releases is
// an accumulator that it has read into registers.  (ptx::mbar_arrive_cluster's release at cluster
// scope waits for the stores before it, 2000 clocks a tile.)
__device__ __forceinline__ void arrive_even(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                   ptx::mapa_shared(ptx::smem_u32(bar), 0))
               : "memory");
}

struct Abort {
  volatile int* flag;          // ends every wait of this CTA
  uint32_t peer_flag;          // ... of the pair's other CTA (shared::cluster address)
  unsigned int* status;        // sticky word of the workspace
};
__device__ __forceinline__ void give_up(const Abort& ab, unsigned int bit) {
  *ab.flag = 1;
  ptx::st_cluster_u32(ab.peer_flag, 1u);
  atomicOr(ab.status, bit);
}

template <int kBN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ LinearMaps M, const __grid_constant__ LinearLaunch L) {
  using C = Cfg<kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const staging = ring + C::kStages * C::kStageBytes;
  uint64_t* const full = reinterpret_cast<uint64_t*>(staging + C::kStagingBytes);
  uint64_t* const empty = full + C::kStages;
  uint64_t* const acc_full = empty + C::kStages;
  uint64_t* const acc_empty = acc_full + 2;
  uint64_t* const drain = acc_empty + 2;
  uint64_t* const in_bar = drain + 1;                 // per epilogue warp and slot
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(in_bar + kEpiWarps * kSlots);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  ptx::griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&full[s], 1);                    // the even CTA's expect_tx (+ all bytes)
      ptx::mbar_init(&empty[s], 1);                   // the pair's commit
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&acc_full[s], 1);
      ptx::mbar_init(&acc_empty[s], 2 * kEpiWarps);   // both CTAs' epilogue warps
    }
    ptx::mbar_init(drain, 1);
    for (int i = 0; i < kEpiWarps * kSlots; ++i) ptx::mbar_init(&in_bar[i], 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, C::kTmemCols);
    ptx::tmem_relinquish_pair();
  } else if (warp == 0 && ptx::elect_one()) {
    for (int p = 0; p < L.n_prob; ++p) {
      ptx::prefetch_tmap(&M.a[p]);
      ptx::prefetch_tmap(&M.b[p]);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();       // both CTAs' barriers exist before either's copies signal them
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();       // the kernel before: inputs, and the workspace it may still use
  Abort ab;
  ab.flag = abort_flag;
  ab.peer_flag = ptx::mapa_shared(ptx::smem_u32(const_cast<const int*>(abort_flag)),
                                  static_cast<uint32_t>(rank ^ 1));
  ab.status = L.status;
  // An earlier failure on this workspace: the products run, and nothing is stored.  (Every warp
  // reads the word beside its first steps: a decision common to the pair before them cost each
  // launch 0.6 us.)  Waits that find it set later give up; after an earlier failure they do not
  // look at it, so that the pair ends in step.
  const bool failed = ptx::status_set(ab.status);
  const unsigned int* const watched = failed ? nullptr : ab.status;
  if (warp == 0) {
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    // (the warp walks in step and an elected lane issues, as for the products: from a branch on
    // a lane index the copies of a step took longer to issue than its products to run)
    for (int i = first; ok && i < L.items; i += stride) {
      const Item it = decode(L, i);
      const LinearProblem& P = L.prob[it.p];
      const bool a_mn = P.a_mn != 0, b_mn = P.b_mn != 0;
      const CUtensorMap *ma = &M.a[it.p], *mb = &M.b[it.p];
      const int row = (2 * it.pr + rank) * kTileM, col = it.tn * kBN + rank * (kBN / 2);
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        ok = ptx::mbar_wait(&empty[stage], phase ^ 1u, ab.flag, watched);
        __syncwarp();
        if (!ok) break;
        uint8_t* const sa = ring + stage * C::kStageBytes;
        uint8_t* const sb = sa + C::kABytes;
        const uint32_t bar = full0 + stage * 8;
        if (ptx::elect_one()) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          if (a_mn) {            // slabs of 64 rows of the tile x 64 deep
            ptx::tma_load_3d_pair(sa, ma, row, kb * kTileK, 0, bar);
            ptx::tma_load_3d_pair(sa + 8192, ma, row + 64, kb * kTileK, 0, bar);
          } else {
            ptx::tma_load_3d_pair(sa, ma, kb * kTileK, row, 0, bar);
          }
          if (b_mn) {
#pragma unroll
            for (int q = 0; q < kBN / 128; ++q)
              ptx::tma_load_3d_pair(sb + q * 8192, mb, col + q * 64, kb * kTileK, 0, bar);
          } else {
            ptx::tma_load_3d_pair(sb, mb, kb * kTileK, col, 0, bar);
          }
        }
        __syncwarp();
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) give_up(ab, kErrTimeoutProducer);
    // before exit every copy has landed and no commit is on its way to this CTA: the
    // products have released every armed stage (after a failure, one bounded window)
    const uint64_t t0 = ptx::globaltimer();
    for (int s = 0; s < C::kStages; ++s) {
      if (!(armed & (1u << s))) continue;
      const uint64_t spent = ptx::globaltimer() - t0;
      if (spent >= ptx::kWaitTimeoutNs ||
          !ptx::mbar_wait(&empty[s], (armed_parity >> s) & 1u, nullptr, nullptr,
                          ptx::kWaitTimeoutNs - spent)) {
        give_up(ab, kErrTimeoutDrain);
        break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = first; ok && i < L.items; i += stride) {
        const Item it = decode(L, i);
        const LinearProblem& P = L.prob[it.p];
        const bool a_mn = P.a_mn != 0, b_mn = P.b_mn != 0;
        const uint32_t idesc = ptx::idesc_bf16(2 * kTileM, kBN, b_mn, a_mn);
        // both CTAs' epilogues have read this accumulator
        ok = ptx::mbar_wait(&acc_empty[acc], acc_phase ^ 1u, ab.flag, watched);
        __syncwarp();
        ptx::tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * kBN);
        for (int kb = it.kb0; ok && kb < it.kb1; ++kb) {
          ok = ptx::mbar_wait(&full[stage], phase, ab.flag, watched);
          __syncwarp();
          if (!ok) break;
          const uint32_t sa = ptx::smem_u32(ring + stage * C::kStageBytes);
          const uint32_t sb = sa + C::kABytes;
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k) {
              // K-major: a K = 16 slice is 32 B on, 8-row groups 1024 B apart.  MN-major:
              // a slice is 16 rows = 2048 B on, 64-column slabs 8192 B apart.
              const uint64_t da = a_mn ? ptx::smem_desc_sw128(sa + k * 2048, 8192, 1024)
                                       : ptx::smem_desc_sw128(sa + k * 32, 16, 1024);
              const uint64_t db = b_mn ? ptx::smem_desc_sw128(sb + k * 2048, 8192, 1024)
                                       : ptx::smem_desc_sw128(sb + k * 32, 16, 1024);
              ptx::mma_bf16_pair(d, da, db, idesc, kb != it.kb0 || k != 0 ? 1u : 0u);
            }
            ptx::mma_commit_pair(&empty[stage]);
            if (kb + 1 == it.kb1) ptx::mma_commit_pair(&acc_full[acc]);
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && lane == 0) give_up(ab, kErrTimeoutMma);
      __syncwarp();
      // every product has completed before TMEM is freed
      if (ptx::elect_one()) ptx::mma_commit_pair(drain, 1);
      __syncwarp();
      if (!ptx::mbar_wait(drain, 0, nullptr) && lane == 0) give_up(ab, kErrTimeoutDrain);
      __syncwarp();
    }
  } else {
    const int e = warp - 2, quarter = warp & 3, half = e >> 2;
    uint8_t* const slots = staging + e * kSlots * kSlotBytes;
    uint64_t* const my_in = in_bar + e * kSlots;
    int acc = 0, slot = 0;
    uint32_t acc_phase = 0, in_par = 0, in_armed = 0;
    const bool skip = failed;
    for (int i = first; i < L.items; i += stride) {
      const Item it = decode(L, i);
      const LinearProblem& P = L.prob[it.p];
      const int i0 = (2 * it.pr + rank) * kTileM + quarter * 32;    // first row of the warp
      const int c0 = it.tn * kBN + half * (kBN / 2);                // first column
      const int units = !skip && i0 < P.m ? min(C::kUnits, max(0, (P.n - c0 + 63) / 64)) : 0;
      const bool split = P.splits > 1;
      const bool has_res = P.has_res != 0 && !split, has_z = P.has_z != 0 && !split;
      auto fetch = [&](int u) {       // the residual's block of unit u into slot u (lane 0)
        ptx::mbar_arrive_expect_tx(&my_in[u], kSlotBytes);
        ptx::tma_load_3d(slots + u * kSlotBytes, &M.res[it.p], c0 + 64 * u, i0, 0, &my_in[u]);
      };
      // Without z both slots are free for this tile's blocks once the last tile's stores have read
      // them: one wait, before the one for the products (each takes 400 clocks, waited for or not).
      if (!has_z || has_res) {
        if (ptx::elect_one()) {
          ptx::bulk_wait_read<0>();
          if (has_res)
            for (int u = 0; u < units && (u == 0 || !has_z); ++u) fetch(u);
        }
        if (has_res) in_armed = units > 0 ? (has_z ? 1u : (1u << units) - 1u) : 0u;
        __syncwarp();
      }
      // the first block's bias travels while the products run, the second's with the first's
      const bool has_bias = P.bias != nullptr && !split;
      uint4 bias[8];
      auto fetch_bias = [&](int j0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = j0 + 8 * q;
          if (c + 8 <= P.n) {
            bias[q] = __ldg(reinterpret_cast<const uint4*>(P.bias + c));
          } else {
            float b[8];
            load8(P.bias, c, P.n, b);
            bias[q] = pack8(b);
          }
        }
      };
      if (has_bias && units > 0) fetch_bias(c0);
      bool ok = ptx::mbar_wait(&acc_full[acc], acc_phase, ab.flag, watched);
      __syncwarp();
      ptx::tc_fence_after();
      const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                          static_cast<uint32_t>(acc * kBN + half * (kBN / 2));
#pragma unroll 1
      for (int u = 0; ok && u < units; ++u) {
        float z[64];
        {
          uint32_t lo[32], hi[32];
          ptx::tmem_ld32x2_sync(t0 + u * 64, t0 + u * 64 + 32, lo, hi);
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            z[q] = __uint_as_float(lo[q]);
            z[32 + q] = __uint_as_float(hi[q]);
          }
        }
        if (split) {
          // this split's sums, four columns of 32 rows at a time: 512 B a store
          float4* const out = reinterpret_cast<float4*>(P.parts) +
              ((static_cast<size_t>(i - P.item_begin) * 2 + rank) * kEpiWarps + e) *
                  (C::kUnits * 512) + u * 512 + lane;
#pragma unroll
          for (int q = 0; q < 16; ++q)
            __stcg(out + q * 32, make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]));
          continue;
        }
        const int j0 = c0 + u * 64;
        // A TMA store writes whole units of 16 bytes: columns up to the next multiple of 8.  The
        // block at the end of a row that ends inside a unit is stored by the lanes.
        const bool ragged = j0 + 64 > P.n && (P.n & 7) != 0;
        auto store_row = [&](__nv_bfloat16* to, long long stride) {
          if (i0 + lane >= P.m) return;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = z[8 * q + j];
            store8(to + (i0 + lane) * stride, j0 + 8 * q, P.n, v);
          }
        };
        if (has_bias) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float b[8];
            unpack8(bias[q], b);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[8 * q + j] += b[j];
          }
          if (u + 1 < units) fetch_bias(j0 + 64);
        }
        if (has_z && ragged) {
          store_row(P.z, P.z_stride);
        } else if (has_z) {
          const int zs = has_res ? 1 : slot;
          if (ptx::elect_one()) {
            // the slot's last store has read it (with a residual only slot 1 is free)
            if (has_res) ptx::bulk_wait_read<0>();
            else ptx::bulk_wait_read<kSlots - 1>();
          }
          __syncwarp();
          stage_row(slots + zs * kSlotBytes, lane, z);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (ptx::elect_one()) {
            ptx::tma_store_3d(&M.z[it.p], j0, i0, 0, slots + zs * kSlotBytes);
            ptx::bulk_commit();
          }
          if (!has_res) slot ^= 1;
        }
        activate(z, P.act);
        int ys = has_z ? slot : u;
        if (has_res) {
          ys = has_z ? 0 : u;
          ok = ptx::mbar_wait(&my_in[ys], (in_par >> ys) & 1u, ab.flag, watched);
          __syncwarp();
          if (!ok) break;
          in_par ^= 1u << ys;
          in_armed &= ~(1u << ys);
          const uint8_t* blk = slots + ys * kSlotBytes;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float r[8];
            unpack8(*reinterpret_cast<const uint4*>(blk + sw128(lane, 8 * q)), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[8 * q + j] += r[j];
          }
        } else if (has_z) {
          if (ptx::elect_one()) ptx::bulk_wait_read<kSlots - 1>();
          __syncwarp();
        }
        if (ragged) {
          store_row(P.out, P.out_stride);
        } else {
          stage_row(slots + ys * kSlotBytes, lane, z);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (ptx::elect_one()) {
            ptx::tma_store_3d(&M.out[it.p], j0, i0, 0, slots + ys * kSlotBytes);
            ptx::bulk_commit();
          }
          if (has_z && !has_res) slot ^= 1;
        }
        if (has_res && has_z && u + 1 < units) {
          if (ptx::elect_one()) {
            ptx::bulk_wait_read<0>();
            ptx::mbar_arrive_expect_tx(&my_in[0], kSlotBytes);
            ptx::tma_load_3d(slots, &M.res[it.p], j0 + 64, i0, 0, &my_in[0]);
          }
          in_armed |= 1u;
          __syncwarp();
        }
      }
      if (!ok) {
        if (lane == 0) give_up(ab, kErrTimeoutEpilogue);
        // copies still in flight land within microseconds
        for (int s = 0; s < kSlots; ++s)
          if (in_armed & (1u << s)) ptx::mbar_wait(&my_in[s], (in_par >> s) & 1u, nullptr);
        __syncwarp();
        break;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (ptx::elect_one()) arrive_even(&acc_empty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (ptx::elect_one()) ptx::bulk_wait_read<0>();
    __syncwarp();
  }
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();       // no CTA leaves while the other may still write to it
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------ finish
// What a split product leaves: the sums of the splits in order, then the epilogue.  A warp
// takes 32 rows x 16 columns of a tile (the layout in which the splits stored them), a lane
// one row's 16 columns.  Also the last level of the bias' gradient: a warp 32 columns.
__global__ void __launch_bounds__(256) linear_finish_kernel(const __grid_constant__ LinearLaunch L) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(L.status)) return;
  const int lane = threadIdx.x & 31;
  long long task = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int per_tile = L.bn / 2;                      // 256 x bn / (32 x 16)
  for (int p = 0; p < L.n_prob; ++p) {
    const LinearProblem& P = L.prob[p];
    if (P.splits <= 1) continue;
    const int tiles = P.tiles_m * P.tiles_n;
    const long long tasks = static_cast<long long>(tiles) * per_tile;
    if (task >= tasks) {
      task -= tasks;
      continue;
    }
    const int units = L.bn / 128;                     // 64-column blocks of an epilogue warp
    const int tile = static_cast<int>(task / per_tile);
    int w = static_cast<int>(task - static_cast<long long>(tile) * per_tile);
    const int part = w & 3;                           // 16 of the block's 64 columns
    w >>= 2;
    const int u = w % units, e = (w / units) % kEpiWarps, rank = w / units / kEpiWarps;
    const Item it = decode(L, P.item_begin + tile);
    const int quarter = (e + 2) & 3, half = e >> 2;
    const int i = (2 * it.pr + rank) * kTileM + quarter * 32 + lane;
    const int j = it.tn * L.bn + half * (L.bn / 2) + u * 64 + part * 16;
    if (i >= P.m || j >= P.n) return;
    const float4* in = reinterpret_cast<const float4*>(P.parts) +
        ((static_cast<size_t>(tile) * 2 + rank) * kEpiWarps + e) * (units * 512) + u * 512 +
        part * 128 + lane;
    const size_t step = static_cast<size_t>(tiles) * 2 * kEpiWarps * units * 512;
    float z[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) z[q] = 0.f;
#pragma unroll 4
    for (int s = 0; s < P.splits; ++s) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 x = __ldcg(in + s * step + q * 32);
        z[4 * q] += x.x; z[4 * q + 1] += x.y; z[4 * q + 2] += x.z; z[4 * q + 3] += x.w;
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v[8], x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = z[8 * q + k];
      const int c = j + 8 * q;
      if (c >= P.n) break;
      if (P.bias != nullptr) {
        load8(P.bias, c, P.n, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += x[k];
      }
      if (P.has_z) store8(P.z + i * P.z_stride, c, P.n, v);
      activate(v, P.act);
      if (P.has_res) {
        // (not through the read-only path: the output may be the residual itself)
        const __nv_bfloat16* row = P.res + i * P.res_stride;
        if (c + 8 <= P.n) {
          unpack8(*reinterpret_cast<const uint4*>(row + c), x);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = c + k < P.n ? __bfloat162float(row[c + k]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += x[k];
      }
      store8(P.out + i * P.out_stride, c, P.n, v);
    }
    return;
  }
  if (L.dbias != nullptr && task * 32 < L.db_n) {
    const int j = static_cast<int>(task) * 32 + lane;
    if (j >= L.db_n) return;
    float s = 0.f;
#pragma unroll 8
    for (int c = 0; c < L.db_chunks; ++c) s += __ldcg(L.db_parts + static_cast<size_t>(c) * L.db_n + j);
    L.dbias[j] = __float2bfloat16_rn(s);
  }
}

// ------------------------------------------------------------ dz and the bias' gradient
// dz = dy act'(z), rounded to bf16 for the products, and the columns' sums of the unrounded
// dz over the rows of a chunk.  Bound by HBM: 8192 x 8192 (403 MB) takes 66 us, 6.1 TB/s.
// (z comes in as it was stored, in bf16: its half step and dz's each add as much to a
// gradient's error as the gradient's own rounding.  fp32 would double the largest activation
// that a training step keeps.  relu^2's z could be had from its output at half that rounding.)  A block takes 256 columns (8 a lane) and a chunk of rows,
// a warp every eighth row of it; the chunks are added by linear_finish_kernel.
constexpr int kDzRows = 4;                  // rows of a warp in flight
__global__ void __launch_bounds__(256) linear_dz_kernel(const __grid_constant__ LinearDz D) {
  __shared__ float s_sum[8][256];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (ptx::status_set(D.status)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lane * 8;
  const int r0 = blockIdx.y * D.chunk, r1 = min(D.rows, r0 + D.chunk);
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = 0.f;
  const bool whole = c + 8 <= D.cols;
  if (c < D.cols) {
    for (int r = r0 + warp; r < r1; r += 8 * kDzRows) {
      uint4 g[kDzRows], z[kDzRows];
      if (whole) {
#pragma unroll
        for (int i = 0; i < kDzRows; ++i) {
          if (r + 8 * i >= r1) break;
          g[i] = __ldg(reinterpret_cast<const uint4*>(D.dy + (r + 8 * i) * D.dy_stride + c));
          if (D.act != MUON_ACT_NONE)
            z[i] = __ldg(reinterpret_cast<const uint4*>(D.z + (r + 8 * i) * D.z_stride + c));
        }
      }
#pragma unroll
      for (int i = 0; i < kDzRows; ++i) {
        const long long row = r + 8 * i;
        if (row >= r1) break;
        float v[8], x[8];
        if (whole) unpack8(g[i], v);
        else load8(D.dy + row * D.dy_stride, c, D.cols, v);
        if (D.act != MUON_ACT_NONE) {
          if (whole) unpack8(z[i], x);
          else load8(D.z + row * D.z_stride, c, D.cols, x);
          times_slope(v, x, D.act);
          store8(D.dz + row * D.dz_stride, c, D.cols, v);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += v[k];
      }
    }
  }
  if (D.parts == nullptr) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) s_sum[warp][lane * 8 + k] = sum[k];
  __syncthreads();
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= D.cols) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += s_sum[w][threadIdx.x];
  __stcg(D.parts + static_cast<size_t>(blockIdx.y) * D.cols + j, s);
}

// ------------------------------------------------------------ a few tokens
// y of up to kTokenMax tokens on the CUDA cores: a warp holds kRows rows of W, a lane 8
// consecutive columns of them at a time, and the tokens' x come from L1.  `ks` warps of a block
// share the rows and split the columns; their sums meet in shared memory.  Bound by reading W:
// 11008 x 4096 (90 MB) takes 16.9 us for one token and 17.2 for two, 5.3 TB/s; what is missing
// to the copy's rate is the start, of which the prefetch hides 0.6 to 3.7 us (17.5 and 21.0
// without; with 4 steps ahead 22.7).  For 3 and 4 tokens 24.6 us (tensor cores: 26), for 8
// it was 46.7, so that these go to the tensor cores.
constexpr int kTokenWarps = 8;              // of a block, at most
constexpr int kTokenRows = 4;               // (with 2: 22.7 us instead of 17.5 at the size below)
constexpr int kTokenAhead = 2;              // steps of W that are asked into L2 ahead
template <int kT>
__global__ void __launch_bounds__(32 * kTokenWarps)
    linear_token_kernel(const __grid_constant__ LinearToken P) {
  constexpr int kRows = kTokenRows;
  __shared__ float s_sum[kTokenWarps][kRows][kT];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (blockDim.x >> 5) / P.ks;           // row groups of a block
  const int row0 = (blockIdx.x * per + warp / P.ks) * kRows;
  const int part = warp % P.ks;
  uint64_t acc[kRows][kT];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[r][t] = 0;
  const int whole = P.k & ~7;
  const __nv_bfloat16* wp[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)                     // (rows past the last repeat it)
    wp[r] = P.w + min(row0 + r, P.n - 1) * P.w_stride;
  // the first of W into L2 while the kernel before ends (its stores to W, if any, are seen by
  // the loads, which wait for it)
#pragma unroll
  for (int i = 0; i < kTokenAhead; ++i) {
    const int c = (part * 32 + lane) * 8 + i * P.ks * 256;
    if (c >= whole) break;
#pragma unroll
    for (int r = 0; r < kRows; ++r) asm volatile("prefetch.global.L2 [%0];" ::"l"(wp[r] + c));
  }
  ptx::griddep_wait();
  const bool failed = ptx::status_set(P.status);      // (nothing is stored then)
#pragma unroll 2
  for (int c = (part * 32 + lane) * 8; c < whole; c += P.ks * 256) {
    uint4 w[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) w[r] = __ldcs(reinterpret_cast<const uint4*>(wp[r] + c));
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(P.x + min(t, P.tokens - 1) * P.x_stride + c));
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      uint64_t xp[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) xp[k] = ptx::pair(bf_lo(xs[k]), bf_hi(xs[k]));
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t ws[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          acc[r][t] = ptx::fma2(ptx::pair(bf_lo(ws[k]), bf_hi(ws[k])), xp[k], acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const float2 a = ptx::unpair(acc[r][t]);
      float s = a.x + a.y;
      // the last columns of a width that is no multiple of 8
      if (part == 0 && whole + lane < P.k)
        s = fmaf(__bfloat162float(wp[r][whole + lane]),
                 __bfloat162float(P.x[min(t, P.tokens - 1) * P.x_stride + whole + lane]), s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) s_sum[warp][r][t] = s;
    }
  }
  __syncthreads();
  if (failed) return;
  // one thread a result
  for (int i = threadIdx.x; i < per * kRows * P.tokens; i += blockDim.x) {
    const int t = i / (per * kRows), rr = i - t * (per * kRows);
    const int grp = rr / kRows, r = rr - grp * kRows;
    const int j = (blockIdx.x * per + grp) * kRows + r;
    if (j >= P.n) continue;
    float z = 0.f;
    for (int s = 0; s < P.ks; ++s) z += s_sum[grp * P.ks + s][r][t];
    if (P.bias != nullptr) z += __bfloat162float(P.bias[j]);
    if (P.z != nullptr) P.z[t * P.z_stride + j] = __float2bfloat16_rn(z);
    float y[1] = {z};
    activate(y, P.act);
    z = y[0];
    if (P.res != nullptr) z += __bfloat162float(P.res[t * P.res_stride + j]);
    P.out[t * P.out_stride + j] = __float2bfloat16_rn(z);
  }
}

// ------------------------------------------------------------ launchers
template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, int cluster,
                             cudaStream_t s, const A&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Pairs that fit on the current device at once (one CTA an SM), asked once a device.
template <int kBN>
cudaError_t pairs_of_device(int sms, int* out) {
  static int cache[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (cache[dev] == 0) {
    e = cudaFuncSetAttribute(linear_gemm_kernel<kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<kBN>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<kBN>::kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2 * (sms / 2));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, linear_gemm_kernel<kBN>, &cfg);
    if (e != cudaSuccess) return e;
    cache[dev] = n < 1 ? 1 : n;
  }
  *out = cache[dev];
  return cudaSuccess;
}

template <int kBN>
cudaError_t launch_gemm_bn(const LinearMaps& m, const LinearLaunch& l, int sms, cudaStream_t s) {
  int n = 0;
  const cudaError_t e = pairs_of_device<kBN>(sms, &n);
  if (e != cudaSuccess) return e;
  return launch_dependent(linear_gemm_kernel<kBN>, dim3(2 * std::min(n, l.items)), kThreads,
                          Cfg<kBN>::kSmem, 2, s, m, l);
}

}  // namespace

cudaError_t launch_linear(const LinearMaps& m, const LinearLaunch& l, int sms, cudaStream_t s) {
  return l.bn == 256 ? launch_gemm_bn<256>(m, l, sms, s) : launch_gemm_bn<128>(m, l, sms, s);
}

cudaError_t launch_linear_finish(const LinearLaunch& l, cudaStream_t s) {
  long long warps = l.dbias != nullptr ? (l.db_n + 31) / 32 : 0;
  for (int p = 0; p < l.n_prob; ++p)
    if (l.prob[p].splits > 1)
      warps += 1ll * l.prob[p].tiles_m * l.prob[p].tiles_n * (l.bn / 2);
  return launch_dependent(linear_finish_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), 256,
                          0, 1, s, l);
}

cudaError_t launch_linear_dz(const LinearDz& d, cudaStream_t s) {
  return launch_dependent(linear_dz_kernel,
                          dim3((d.cols + 255) / 256, d.rows / d.chunk + (d.rows % d.chunk != 0)),
                          256, 0, 1,
                          s, d);
}

template <int kT>
static cudaError_t launch_token(LinearToken p, int sms, cudaStream_t s) {
  // as many warps on the rows' columns as it takes to give every SM 16 warps
  constexpr int kRows = kTokenRows;
  const int groups = (p.n + kRows - 1) / kRows;
  p.ks = 1;
  while (p.ks < kTokenWarps && groups * p.ks < 16 * sms && p.ks * 256 < p.k) p.ks *= 2;
  const int warps = std::max(4, p.ks), per = warps / p.ks;
  return launch_dependent(linear_token_kernel<kT>, dim3((groups + per - 1) / per), 32 * warps, 0, 1,
                          s, p);
}

cudaError_t launch_linear_token(const LinearToken& p, int sms, cudaStream_t s) {
  switch (p.tokens) {
    case 1: return launch_token<1>(p, sms, s);
    case 2: return launch_token<2>(p, sms, s);
    default: return launch_token<4>(p, sms, s);
  }
}

}  // namespace muon
