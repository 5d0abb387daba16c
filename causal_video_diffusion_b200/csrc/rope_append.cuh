// rope_append.cuh -- where an element of a chunk lives: index decode shared by the append kernels
// (bf16 and 8-bit caches).
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace unstep {

__device__ __forceinline__ uint4 ld_plain(const void *p) {
  return *reinterpret_cast<const uint4 *>(p);
}

struct Item {
  long long e;       // element offset of the 8-channel vector in q/k/v (the activations)
  long long ce;      // element offset in the caches
  float2 cs[4];      // cos/sin of its 4 channel pairs
};

// Where item `it` (one 8-channel vector of one (stream, token, head)) lives, and its coefficients.
// All index arithmetic is 32-bit (items < 2^31, checked on the host) with multiply-high division.
// Returns false only in the debug build, when an index falls outside its tensor (the item is
// then skipped and the error word set).
// kHeads > 0: items stand for kHeads heads each, H / kHeads apart (div_h divides by H / kHeads), are
// located at the first, and run through a head's tokens before the next head's.
template <int D, int kHeads = 0>
__device__ __forceinline__ bool locate(const RopeAppendParams &p, uint32_t it, Item &m) {
  constexpr int kLogV = (D == 128) ? 4 : 3;  // 16-byte vectors per head row: D / 8
  const uint32_t c8 = it & ((1u << kLogV) - 1);
  const uint32_t r = it >> kLogV;
  uint32_t b, h, l;
  if constexpr (kHeads == 0) {                // r = (b*L + l)*H + h
    const uint32_t bl = fdiv(r, p.div_h);
    h = r - bl * static_cast<uint32_t>(p.H);
    b = fdiv(bl, p.div_l);
    l = bl - b * static_cast<uint32_t>(p.L);
  } else {                                    // r = (b*H/kHeads + h)*L + l
    const uint32_t bh = fdiv(r, p.div_l);
    l = r - bh * static_cast<uint32_t>(p.L);
    b = fdiv(bh, p.div_h);
    h = bh - b * (static_cast<uint32_t>(p.H) / kHeads);
  }
  const uint32_t i = fdiv(l, p.div_tf);
  const uint32_t tok = l - i * static_cast<uint32_t>(p.Tf);
  const uint32_t y = fdiv(tok, p.div_wg);
  const uint32_t x = tok - y * static_cast<uint32_t>(p.Wg);
  const int f = p.frame_idx + static_cast<int>(i);
  int slot = p.slot0 + static_cast<int>(i);   // i < frames <= cap: one wrap at most
  if (slot >= p.cap) slot -= p.cap;
  // q, k, v: the shard's stream and head within the activations (it * 8 when unsharded)
  m.e = kHeads > 0 || p.sharded
            ? ((static_cast<long long>(p.b0) + b) * p.L + l) * p.act_H * D +
                  (static_cast<long long>(p.h0) + h) * D + c8 * 8
            : static_cast<long long>(it) * 8;
  m.ce = ((static_cast<long long>(b) * p.H + h) * p.rows + static_cast<long long>(slot) * p.Tf +
          tok) * D + c8 * 8;
  if (kDebugChecks) {
    const long long n_act = static_cast<long long>(p.act_B) * p.L * p.act_H * D;
    const long long n_cache = static_cast<long long>(p.B) * p.H * p.rows * D;
    // from the item's first head to its last
    const long long more = kHeads > 0 ? (kHeads - 1) * static_cast<long long>(p.H / kHeads) : 0;
    const bool ok = b < static_cast<uint32_t>(p.B) && h < static_cast<uint32_t>(p.H) &&
                    i < static_cast<uint32_t>(p.frames) && y < static_cast<uint32_t>(p.Hg) &&
                    slot >= 0 && slot < p.cap && f >= 0 && f < p.max_pos_t && m.e >= 0 &&
                    m.e + more * D + 8 <= n_act && m.ce >= 0 &&
                    m.ce + more * p.rows * D + 8 <= n_cache;
    if (!debug_check(ok, p.dev_error)) return false;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int pr = static_cast<int>(c8) * 4 + u;  // channel pair index
    const float2 *src;
    if (pr < p.half_t) {
      src = p.tab_t + f * p.half_t + pr;
    } else if (pr < p.half_t + p.half_h) {
      src = p.tab_h + static_cast<int>(y) * p.half_h + (pr - p.half_t);
    } else {
      src = p.tab_w + static_cast<int>(x) * p.half_w + (pr - p.half_t - p.half_h);
    }
    m.cs[u] = __ldg(src);  // the tables are written by the cache's initialisation alone
  }
  return true;
}

}  // namespace unstep
