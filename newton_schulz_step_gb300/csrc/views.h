// views.h -- what the host sides of the entry points share: alignment, the workspace's
// check, and whether two strided views reach the same bytes.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "internal.h"
#include "workspace_turn.h"

namespace muon {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline muon_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < need)
    return MUON_ERR_WORKSPACE;
  return MUON_OK;
}

// Bytes that a call reads or writes: `len` at every (token, head).
struct Rows {
  uintptr_t at;
  long long ts, hs, len;                    // bytes
  int tokens, heads;
};
inline Rows rows_of(const muon_heads& v, int tokens, int heads, int dim, int size) {
  return {reinterpret_cast<uintptr_t>(v.data), v.token_stride * size, v.head_stride * size,
          1ll * dim * size, tokens, heads};
}
inline Rows rows_of(const float* p, long long n) {
  return {reinterpret_cast<uintptr_t>(p), 0, 0, n * 4, 1, 1};
}
inline uintptr_t end_of(const Rows& r) { return r.at + r.ts * (r.tokens - 1) + r.hs * (r.heads - 1) + r.len; }
inline long long floor_div(long long a, long long b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// Whether the two share a byte.  Views that interleave (the columns of one fused tensor) have
// one token stride; of others that reach into each other's range, and of more heads than a
// check should cost, the answer is yes.
inline bool overlap(const Rows& a, const Rows& b) {
  if (a.at >= end_of(b) || b.at >= end_of(a)) return false;
  if (a.tokens > 1 && b.tokens > 1 && a.ts != b.ts) return true;
  const long long ts = std::max(1ll, a.tokens > 1 ? a.ts : b.ts);
  const long long apart = static_cast<long long>(a.at - b.at);
  // all heads of a token as one piece: a's piece lies between two of b's
  const long long gap = apart - floor_div(apart, ts) * ts;
  if (gap >= b.hs * (b.heads - 1) + b.len && gap + a.hs * (a.heads - 1) + a.len <= ts)
    return false;
  if (1ll * a.heads * b.heads > 1 << 16) return true;
  const bool one_stride = a.hs == b.hs;      // then head i - j of a over head 0 of b says it all
  for (int i = 0; i < a.heads; ++i)
    for (int j = 0; j < b.heads; ++j) {
      if (one_stride && i > 0 && j > 0) break;
      // tokens d apart are off + d ts apart; they meet if -a.len < off + d ts < b.len
      const long long off = apart + i * a.hs - j * b.hs;
      const long long lo = floor_div(-a.len - off, ts) + 1, hi = -floor_div(off - b.len, ts) - 1;
      if (std::max(lo, 1ll - b.tokens) <= std::min(hi, a.tokens - 1ll)) return true;
    }
  return false;
}
inline bool same_rows(const Rows& a, const Rows& b) {
  return a.at == b.at && (a.tokens == 1 || a.ts == b.ts) && (a.heads == 1 || a.hs == b.hs);
}
// No output shares a byte with an input or with another output.
inline bool apart(std::initializer_list<Rows> outputs, std::initializer_list<Rows> inputs) {
  for (const Rows* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Rows& x : inputs)
      if (overlap(*o, x)) return false;
    for (const Rows* p = outputs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return false;
  }
  return true;
}

}  // namespace muon
