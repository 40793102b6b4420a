// linear_api.cu -- host side of the products with a weight matrix declared in
// include/muon_gb300.h: argument checks, how a product is cut into tiles and splits,
// tensor maps, launches.
//
// Everything is enqueued on the caller's stream; nothing here synchronises or
// allocates device memory.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "views.h"

using namespace muon;

namespace {

constexpr int kMaxFeatures = 1 << 20;
constexpr int kMaxTokens = INT_MAX - 65536;
constexpr int kMaxItems = 1 << 30;
constexpr int kDzChunksMax = 128;

int cdiv(int x, int a) { return x / a + (x % a != 0); }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool matrix_ok(muon_matrix* v, int rows, int cols) {
  if (!v->data || !aligned16(v->data)) return false;
  if (rows == 1) v->row_stride = (cols + 7) / 8 * 8;
  constexpr long long kMaxStride = 1ll << 38;   // below 2^40 bytes (tensor maps)
  return v->row_stride >= cols && v->row_stride < kMaxStride && v->row_stride % 8 == 0;
}
Rows rows_of(const muon_matrix& v, int rows, int cols) {
  return {reinterpret_cast<uintptr_t>(v.data), v.row_stride * 2, 0, 2ll * cols, rows, 1};
}
__nv_bfloat16* ptr(const muon_matrix& v) { return static_cast<__nv_bfloat16*>(v.data); }

bool spec_ok(const muon_linear_spec* s) {
  return s && s->tokens >= 0 && s->tokens <= kMaxTokens && s->in_features >= 1 &&
         s->out_features >= 1 && s->in_features <= kMaxFeatures &&
         s->out_features <= kMaxFeatures && s->activation >= MUON_ACT_NONE &&
         s->activation <= MUON_ACT_GELU && aligned16(s->bias);
}

// ------------------------------------------------------------ tiles and splits
struct Product {
  int m, n, k;
};

// Estimated clocks of a call's launches with `count` products, tiles bn wide and the given splits.
// A 64-deep step of a 256 x 256 tile takes the tensor cores 512 clocks (530 measured); of a
// 256 x 128 tile half that, but its operands, 24 KB a CTA, were not seen to arrive in less than
// 420.  A tile takes its epilogue 8 clocks a column if the products are over sooner.  Sums of
// splits: a launch, their way to L2 and back, and a trip to L2 for every four of them.
// (Swept over both widths and 1 to 16 splits on 16 shapes of 33 to 8192 tokens, 64 to 11008 wide:
// the choice was the fastest or within 14 % of it.)
double plan_clocks(const Product* p, int count, int bn, const int* splits) {
  const double step = bn == 256 ? 530.0 : 420.0, fixed = 2500.0;
  double work = 0.0, longest = 0.0, finish = 0.0, waves = 0.0;
  for (int i = 0; i < count; ++i) {
    const double tiles = 1.0 * cdiv(p[i].m, 256) * cdiv(p[i].n, bn);
    const double len = std::max(cdiv(cdiv(p[i].k, kTileK), splits[i]) * step, 8.0 * bn);
    const double items = tiles * splits[i];
    work += items * len;
    longest = std::max(longest, len);
    waves += std::ceil(items / kLinearPairs) * len;
    if (splits[i] > 1)
      finish = std::max(finish, 5500.0 + 300.0 * splits[i]) + 8.0 / 6000.0 * splits[i] * p[i].m * p[i].n;
  }
  // one product: whole waves; two: the shorter items fill the last wave of the longer ones
  const double time = count == 1 ? waves : std::max(longest, work / kLinearPairs + 0.5 * longest);
  return time + fixed + finish;
}

struct Plan {
  int bn;
  int splits[2];
  size_t parts[2];                      // bytes of the splits' sums
};

// The cheapest of both tile widths and of a few splits by the estimate above.  A product is
// split only while its items number at most two a pair.
Plan make_plan(const Product* p, int count) {
  static constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64};
  Plan best{256, {1, 1}, {0, 0}};
  double least = -1.0;
  for (int bn : {256, 128}) {
    auto allowed = [&](int i, int s) {
      const long long tiles = 1ll * cdiv(p[i].m, 256) * cdiv(p[i].n, bn);
      return s == 1 || (s <= cdiv(p[i].k, kTileK) && tiles * s <= 2 * kLinearPairs);
    };
    for (int s0 : kSplits) {
      if (!allowed(0, s0)) break;
      for (int s1 : kSplits) {
        if (count == 1 ? s1 > 1 : !allowed(1, s1)) break;
        const int s[2] = {s0, s1};
        const double c = plan_clocks(p, count, bn, s);
        if (least < 0.0 || c < least) {
          least = c;
          best.bn = bn;
          best.splits[0] = s0;
          best.splits[1] = s1;
        }
      }
    }
  }
  for (int i = 0; i < count; ++i)
    if (best.splits[i] > 1)
      best.parts[i] = static_cast<size_t>(best.splits[i]) * cdiv(p[i].m, 256) *
                      cdiv(p[i].n, best.bn) * 256 * best.bn * sizeof(float);
  return best;
}

// [0] dW, whose contraction over the tokens is the longer one as a rule, [1] dx
void backward_products(int tokens, int in, int out, Product (&p)[2]) {
  p[0] = {out, in, tokens};
  p[1] = {tokens, in, out};
}

// The plan of a call, by its sizes.  Looking for one takes several microseconds (two products:
// 450 estimates), so a thread keeps those of the sizes that it met last.
Plan plan_of(int tokens, int in, int out, bool backward) {
  struct Entry {
    int tokens = -1, in, out;
    bool backward;
    Plan plan;
  };
  static thread_local Entry kept[64];
  const unsigned h = (static_cast<unsigned>(tokens) * 2654435761u) ^
                     (static_cast<unsigned>(in) * 40503u) ^ (static_cast<unsigned>(out) * 9176741u);
  Entry& e = kept[((h >> 16) ^ h ^ (backward ? 1u : 0u)) & 63u];
  if (e.tokens != tokens || e.in != in || e.out != out || e.backward != backward) {
    Product p[2] = {{tokens, out, in}, {0, 0, 0}};
    if (backward) backward_products(tokens, in, out, p);
    e.plan = make_plan(p, backward ? 2 : 1);
    e.tokens = tokens;
    e.in = in;
    e.out = out;
    e.backward = backward;
  }
  return e.plan;
}

// Rows of a block of linear_dz_kernel: enough blocks for four an SM, whole sets of 32 rows.
int dz_chunk(int tokens, int out) {
  const int cols = cdiv(out, 256);
  const int chunks = std::min({cdiv(4 * 2 * kLinearPairs, cols), cdiv(tokens, 32), kDzChunksMax});
  return cdiv(cdiv(tokens, std::max(1, chunks)), 32) * 32;
}

size_t forward_bytes(int tokens, int in, int out) {
  if (tokens <= kTokenMax) return kStatusBytes;
  return kStatusBytes + align256(plan_of(tokens, in, out, false).parts[0]);
}
size_t backward_bytes(int tokens, int in, int out) {
  if (tokens == 0) return kStatusBytes;
  const Plan plan = plan_of(tokens, in, out, true);
  return kStatusBytes + align256(plan.parts[0]) + align256(plan.parts[1]) +
         align256(static_cast<size_t>(cdiv(tokens, dz_chunk(tokens, out))) * out * sizeof(float));
}

// Fills problem i of a launch; false if its items are too many.
bool set_problem(LinearLaunch& L, int i, const Product& p, int splits, bool a_mn, bool b_mn) {
  LinearProblem& P = L.prob[i];
  P.m = p.m;
  P.n = p.n;
  P.k_blocks = cdiv(p.k, kTileK);
  P.tiles_m = cdiv(p.m, 256);
  P.tiles_n = cdiv(p.n, L.bn);
  const long long items = 1ll * P.tiles_m * P.tiles_n * splits + L.items;
  if (items > kMaxItems) return false;
  P.splits = splits;
  P.by_tiles = Divisor::of(P.tiles_m * P.tiles_n);
  P.by_band = Divisor::of(kBand * P.tiles_n);
  P.last_band = (P.tiles_m - 1) / kBand;
  P.by_last = Divisor::of(P.tiles_m - P.last_band * kBand);
  P.k_each = P.k_blocks / splits;
  P.k_more = P.k_blocks - P.k_each * splits;
  P.a_mn = a_mn;
  P.b_mn = b_mn;
  P.item_begin = L.items;
  L.items = static_cast<int>(items);
  L.n_prob = i + 1;
  return true;
}

// Operand with `mn` rows of the tile and k deep: stored [mn][k], or [k][mn] where by_rows.
bool operand(CUtensorMap* tm, const muon_matrix& v, int mn, int k, bool by_rows, int box_rows) {
  return by_rows ? matrix_tmap(tm, v, k, mn, 64, 64) : matrix_tmap(tm, v, mn, k, 64, box_rows);
}

}  // namespace

extern "C" {

size_t muon_linear_workspace_bytes(int tokens, int in_features, int out_features) {
  const muon_linear_spec s{tokens, in_features, out_features, MUON_ACT_NONE, nullptr};
  if (!spec_ok(&s)) return 0;
  return std::max(forward_bytes(tokens, in_features, out_features),
                  backward_bytes(tokens, in_features, out_features));
}

muon_status muon_linear(const muon_linear_spec* spec, muon_matrix x, muon_matrix weight,
                        muon_matrix residual, muon_matrix preact, muon_matrix out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!spec_ok(spec)) return MUON_ERR_INVALID_ARG;
    const int t = spec->tokens, k = spec->in_features, n = spec->out_features;
    const bool has_res = residual.data != nullptr, has_z = preact.data != nullptr;
    muon_status s = check_workspace(workspace, workspace_bytes, forward_bytes(t, k, n));
    if (s != MUON_OK) return s;
    if (t == 0) return MUON_OK;
    if (!matrix_ok(&x, t, k) || !matrix_ok(&weight, n, k) || !matrix_ok(&out, t, n) ||
        (has_res && !matrix_ok(&residual, t, n)) || (has_z && !matrix_ok(&preact, t, n)))
      return MUON_ERR_INVALID_ARG;
    const Rows r_out = rows_of(out, t, n), r_x = rows_of(x, t, k), r_w = rows_of(weight, n, k);
    const Rows r_b = {reinterpret_cast<uintptr_t>(spec->bias), 0, 0, 2ll * n, 1, 1};
    auto clashes = [&](const Rows& o) {
      return overlap(o, r_x) || overlap(o, r_w) || (spec->bias && overlap(o, r_b));
    };
    if (clashes(r_out)) return MUON_ERR_INVALID_ARG;
    if (has_res) {
      const Rows r = rows_of(residual, t, n);
      if (!same_rows(r_out, r) && overlap(r_out, r)) return MUON_ERR_INVALID_ARG;
      if (has_z && overlap(rows_of(preact, t, n), r)) return MUON_ERR_INVALID_ARG;
    }
    if (has_z && (clashes(rows_of(preact, t, n)) || overlap(rows_of(preact, t, n), r_out)))
      return MUON_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned int* const status = static_cast<unsigned int*>(workspace);
    const double flops = 2.0 * t * k * n;
    const double bytes = 2.0 * (1.0 * t * k + 1.0 * n * k + 1.0 * t * n * (1 + has_res + has_z));
    // (the crossing: see linear_token_kernel)
    if (t <= kTokenMax) {
      LinearToken p;
      std::memset(&p, 0, sizeof(p));
      p.x = ptr(x);
      p.w = ptr(weight);
      p.bias = static_cast<const __nv_bfloat16*>(spec->bias);
      p.res = ptr(residual);
      p.z = ptr(preact);
      p.out = ptr(out);
      p.x_stride = x.row_stride;
      p.w_stride = weight.row_stride;
      p.res_stride = residual.row_stride;
      p.z_stride = preact.row_stride;
      p.out_stride = out.row_stride;
      p.tokens = t;
      p.n = n;
      p.k = k;
      p.act = spec->activation;
      p.status = status;
      const cudaError_t e = counted_launch(st, MUON_K_LINEAR_TOKEN, flops, bytes,
                                           [&] { return launch_linear_token(p, sms, st); });
      return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
    }
    LinearLaunch L;
    std::memset(&L, 0, sizeof(L));
    const Plan plan = plan_of(t, k, n, false);
    L.bn = plan.bn;
    L.status = status;
    if (!set_problem(L, 0, {t, n, k}, plan.splits[0], false, false)) return MUON_ERR_UNSUPPORTED;
    LinearProblem& P = L.prob[0];
    P.act = spec->activation;
    P.bias = static_cast<const __nv_bfloat16*>(spec->bias);
    P.has_res = has_res;
    P.has_z = has_z;
    P.out = ptr(out);
    P.z = ptr(preact);
    P.res = ptr(residual);
    P.out_stride = out.row_stride;
    P.z_stride = preact.row_stride;
    P.res_stride = residual.row_stride;
    P.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    LinearMaps M;
    std::memset(&M, 0, sizeof(M));
    if (!operand(&M.a[0], x, t, k, false, kTileM) ||
        !operand(&M.b[0], weight, n, k, false, L.bn / 2) ||
        !matrix_tmap(&M.out[0], out, t, n, 64, 32) ||
        (has_res && !matrix_tmap(&M.res[0], residual, t, n, 64, 32)) ||
        (has_z && !matrix_tmap(&M.z[0], preact, t, n, 64, 32)))
      return MUON_ERR_CUDA;
    const WorkspaceTurn turn(P.splits > 1 ? workspace : nullptr);
    cudaError_t e = counted_launch(st, MUON_K_LINEAR, flops, bytes,
                                   [&] { return launch_linear(M, L, sms, st); });
    if (e == cudaSuccess && P.splits > 1)
      e = counted_launch(st, MUON_K_LINEAR_FINISH, 0.0, static_cast<double>(plan.parts[0]),
                         [&] { return launch_linear_finish(L, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

muon_status muon_linear_backward(const muon_linear_spec* spec, muon_matrix dout, muon_matrix x,
                                 muon_matrix weight, muon_matrix preact, muon_matrix dz,
                                 muon_matrix dx, muon_matrix dweight, void* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!spec_ok(spec) || !aligned16(dbias)) return MUON_ERR_INVALID_ARG;
    const int t = spec->tokens, k = spec->in_features, n = spec->out_features;
    const bool act = spec->activation != MUON_ACT_NONE;
    muon_status s = check_workspace(workspace, workspace_bytes, backward_bytes(t, k, n));
    if (s != MUON_OK) return s;
    if (!matrix_ok(&dweight, n, k)) return MUON_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (t == 0) {                              // sums over nothing
      s = device_sms(&sms);
      if (s != MUON_OK) return s;
      if (cudaMemset2DAsync(dweight.data, dweight.row_stride * 2, 0, 2ll * k, n, st) !=
              cudaSuccess ||
          (dbias && cudaMemsetAsync(dbias, 0, 2ll * n, st) != cudaSuccess))
        return MUON_ERR_CUDA;
      return MUON_OK;
    }
    if (!matrix_ok(&dout, t, n) || !matrix_ok(&x, t, k) || !matrix_ok(&weight, n, k) ||
        !matrix_ok(&dx, t, k) || (act && (!matrix_ok(&preact, t, n) || !matrix_ok(&dz, t, n))))
      return MUON_ERR_INVALID_ARG;
    {
      const Rows in[] = {rows_of(dout, t, n), rows_of(x, t, k), rows_of(weight, n, k),
                         act ? rows_of(preact, t, n) : rows_of(dout, t, n)};
      Rows outs[4] = {rows_of(dx, t, k), rows_of(dweight, n, k)};
      int count = 2;
      if (act) outs[count++] = rows_of(dz, t, n);
      if (dbias) outs[count++] = {reinterpret_cast<uintptr_t>(dbias), 0, 0, 2ll * n, 1, 1};
      for (int i = 0; i < count; ++i) {
        for (const Rows& r : in)
          if (overlap(outs[i], r)) return MUON_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
          if (overlap(outs[i], outs[j])) return MUON_ERR_INVALID_ARG;
      }
    }
    s = device_sms(&sms);
    if (s != MUON_OK) return s;
    Product p[2];
    backward_products(t, k, n, p);
    const Plan plan = plan_of(t, k, n, true);
    uint8_t* const base = static_cast<uint8_t*>(workspace) + kStatusBytes;
    const int chunk = dz_chunk(t, n);
    LinearLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.bn = plan.bn;
    L.status = static_cast<unsigned int*>(workspace);
    const muon_matrix g = act ? dz : dout;
    LinearMaps M;
    std::memset(&M, 0, sizeof(M));
    if (!set_problem(L, 0, p[0], plan.splits[0], true, true) ||
        !set_problem(L, 1, p[1], plan.splits[1], false, true))
      return MUON_ERR_UNSUPPORTED;
    const muon_matrix outs[2] = {dweight, dx};
    for (int i = 0; i < 2; ++i) {
      L.prob[i].out = ptr(outs[i]);
      L.prob[i].out_stride = outs[i].row_stride;
      if (!matrix_tmap(&M.out[i], outs[i], p[i].m, p[i].n, 64, 32)) return MUON_ERR_CUDA;
    }
    L.prob[0].parts = reinterpret_cast<float*>(base);
    L.prob[1].parts = reinterpret_cast<float*>(base + align256(plan.parts[0]));
    if (!operand(&M.a[0], g, n, t, true, 0) || !operand(&M.b[0], x, k, t, true, 0) ||
        !operand(&M.a[1], g, t, n, false, kTileM) || !operand(&M.b[1], weight, k, n, true, 0))
      return MUON_ERR_CUDA;
    LinearDz D;
    std::memset(&D, 0, sizeof(D));
    D.dy = ptr(dout);
    D.dy_stride = dout.row_stride;
    D.z = ptr(preact);
    D.z_stride = preact.row_stride;
    D.dz = ptr(dz);
    D.dz_stride = dz.row_stride;
    D.rows = t;
    D.cols = n;
    D.chunk = chunk;
    D.act = spec->activation;
    D.status = L.status;
    if (dbias) {
      D.parts = reinterpret_cast<float*>(base + align256(plan.parts[0]) + align256(plan.parts[1]));
      L.dbias = static_cast<__nv_bfloat16*>(dbias);
      L.db_parts = D.parts;
      L.db_n = n;
      L.db_chunks = cdiv(t, chunk);
    }
    const bool finish = dbias || plan.splits[0] > 1 || plan.splits[1] > 1;
    const WorkspaceTurn turn(finish ? workspace : nullptr);
    cudaError_t e = cudaSuccess;
    if (act || dbias)
      e = counted_launch(st, MUON_K_LINEAR_DZ, 0.0, 2.0 * t * n * (act ? 3 : 1),
                         [&] { return launch_linear_dz(D, st); });
    if (e == cudaSuccess)
      e = counted_launch(st, MUON_K_LINEAR, 4.0 * t * k * n,
                         2.0 * (2.0 * t * n + 2.0 * t * k + 2.0 * n * k),
                         [&] { return launch_linear(M, L, sms, st); });
    if (e == cudaSuccess && finish)
      e = counted_launch(st, MUON_K_LINEAR_FINISH, 0.0,
                         static_cast<double>(plan.parts[0] + plan.parts[1]),
                         [&] { return launch_linear_finish(L, st); });
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

}  // extern "C"
