// rope_append.cu -- fused 3D RoPE + ring-buffer KV-cache append (one launch per chunk).
//
// UnStep paper (arXiv 2609.32518), abstract: the DiT runtime stack applies RoPE from cached
// coefficients and indexes a KV cache that retains a limited temporal window.  This kernel does
// both in one pass over HBM: q, k, v are read once; rotated q goes back in place, rotated k and v
// go to ring slot f mod cap.  The work is pure streaming (6 bf16 tensors of B*L*H*D elements),
// so it is bound by HBM bandwidth: every thread moves 16-byte vectors, a warp covers 512
// contiguous bytes of each input, and the coefficient tables (< 20 KB) stay in L1/L2.  When the
// attention rotates the queries itself (its query prologue), the K/V-only instantiation leaves q
// alone and moves 4 of the 6 streams.
#include <cuda_bf16.h>

#include "internal.h"
#include "rope_append.cuh"

namespace unstep {
namespace {

constexpr int kThreads = 256;
#ifndef UNSTEP_ROPE_ITEMS
#define UNSTEP_ROPE_ITEMS 1
#endif
// K/V-only form: two vectors of each of its two inputs per thread keep as many bytes in flight
#ifndef UNSTEP_ROPE_ITEMS_KV
#define UNSTEP_ROPE_ITEMS_KV 2
#endif
// independent 16-byte vectors (of each input) per thread
template <bool kQ>
constexpr int items_per_thread() { return kQ ? UNSTEP_ROPE_ITEMS : UNSTEP_ROPE_ITEMS_KV; }

// k and v, which no kernel writes while this one runs: it starts after its predecessors have ended.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// kQ: q is rotated in place; without it q is neither read nor written.
template <int D, bool kQ>
__global__ void __launch_bounds__(kThreads) rope_kv_append_kernel(const RopeAppendParams p,
                                                                   uint32_t n_items) {
  constexpr int kItemsPerThread = items_per_thread<kQ>();
  const uint32_t base = blockIdx.x * (kThreads * kItemsPerThread) + threadIdx.x;
  if (blockIdx.x == 0 && threadIdx.x < p.frames) {
    const int f = p.frame_idx + threadIdx.x;
    if (debug_check(f >= 0 && p.cap > 0, p.dev_error)) p.slot_frame[f % p.cap] = f;
  }
  Item m[kItemsPerThread];
  uint4 qv[kItemsPerThread], kv[kItemsPerThread], vv[kItemsPerThread];
  bool live[kItemsPerThread];
#pragma unroll
  for (int u = 0; u < kItemsPerThread; ++u) {
    const uint32_t it = base + u * kThreads;
    live[u] = it < n_items && locate<D>(p, it, m[u]);
    if (live[u]) {
      if (kQ) qv[u] = ld_plain(static_cast<const __nv_bfloat16 *>(p.q) + m[u].e);
      kv[u] = ld_stream(static_cast<const __nv_bfloat16 *>(p.k) + m[u].e);
      vv[u] = ld_stream(static_cast<const __nv_bfloat16 *>(p.v) + m[u].e);
    }
  }
#pragma unroll
  for (int u = 0; u < kItemsPerThread; ++u) {
    if (!live[u]) continue;
    if (kQ) {
      uint4 qo;
      qo.x = rope_rotate_pair(qv[u].x, m[u].cs[0]);
      qo.y = rope_rotate_pair(qv[u].y, m[u].cs[1]);
      qo.z = rope_rotate_pair(qv[u].z, m[u].cs[2]);
      qo.w = rope_rotate_pair(qv[u].w, m[u].cs[3]);
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.q) + m[u].e) = qo;
    }
    uint4 ko;
    ko.x = rope_rotate_pair(kv[u].x, m[u].cs[0]);
    ko.y = rope_rotate_pair(kv[u].y, m[u].cs[1]);
    ko.z = rope_rotate_pair(kv[u].z, m[u].cs[2]);
    ko.w = rope_rotate_pair(kv[u].w, m[u].cs[3]);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.k_cache) + m[u].ce) = ko;
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.v_cache) + m[u].ce) = vv[u];
  }
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeAppendParams &p, cudaStream_t stream) {
  const long long n_items = static_cast<long long>(p.B) * p.L * p.H * (p.D / 8);
  const int items = p.rotate_q ? items_per_thread<true>() : items_per_thread<false>();
  if (n_items >= (1ll << 31) - kThreads * items) return cudaErrorInvalidConfiguration;
  RopeAppendParams q = p;
  q.slot0 = p.frame_idx % p.cap;
  q.div_h = make_fastdiv(static_cast<uint32_t>(p.H));
  q.div_l = make_fastdiv(static_cast<uint32_t>(p.L));
  q.div_tf = make_fastdiv(static_cast<uint32_t>(p.Tf));
  q.div_wg = make_fastdiv(static_cast<uint32_t>(p.Wg));
  const long long per_block = kThreads * items;
  long long blocks = (n_items + per_block - 1) / per_block;
  if (blocks < 1) blocks = 1;
  const uint32_t n = static_cast<uint32_t>(n_items);
  const dim3 gb(static_cast<unsigned>(blocks));
  if (p.D == 128 && p.rotate_q) {
    rope_kv_append_kernel<128, true><<<gb, kThreads, 0, stream>>>(q, n);
  } else if (p.D == 128) {
    rope_kv_append_kernel<128, false><<<gb, kThreads, 0, stream>>>(q, n);
  } else if (p.D == 64 && p.rotate_q) {
    rope_kv_append_kernel<64, true><<<gb, kThreads, 0, stream>>>(q, n);
  } else if (p.D == 64) {
    rope_kv_append_kernel<64, false><<<gb, kThreads, 0, stream>>>(q, n);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace unstep
