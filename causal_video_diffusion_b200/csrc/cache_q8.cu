// cache_q8.cu -- the 8-bit KV cache: fused 3D RoPE, quantisation and ring-buffer append, and the
// rows read back as bf16.
//
// Append: the same streaming pass as the bf16 append (q, k, v read once), with the rotated k and
// the v quantised in registers: the four lanes that hold a 32-channel block share its maximum by
// two shuffles, then every lane writes the eight codes of its vector.  It moves 10 + 1/16 bytes
// for every element of the chunk (q read and written, k and v read in bf16, two codes and their
// share of two scale bytes) where the bf16 append moves 12.  Measured, call after call on three sets of
// inputs: 13.1 us for 4680 tokens of 12 heads of 128 (5.5 TB/s), four such streams 47.6 us (6.1 TB/s).
// Read-back: 6 + 1/16 bytes an element of K and V: 6.4 us for that chunk (its codes in L2), 28.4 us
// for the four (6.1 TB/s).
#include <cuda_bf16.h>

#include "internal.h"
#include "q8.cuh"
#include "rope_append.cuh"

namespace unstep {
namespace {

constexpr int kThreads = 256;        // of the read-back
constexpr int kAppendThreads = 128;  // six blocks an SM, 9 % faster for a chunk than two of 256
constexpr uint32_t kFullMask = 0xFFFFFFFFu;

// k and v, read once.  Not through the read-only path: the kernel is resident while its predecessor
// may still write them, and q_out may be one of them, so the load is coherent and stays before the
// thread's stores.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Rotates eight channels in fp32, unrounded (the codes are the only rounding of k).
__device__ __forceinline__ void rotate8(float (&x)[8], const float2 (&cs)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float a = x[2 * u], b = x[2 * u + 1];
    x[2 * u] = __fmaf_rn(a, cs[u].x, -__fmul_rn(b, cs[u].y));
    x[2 * u + 1] = __fmaf_rn(a, cs[u].y, __fmul_rn(b, cs[u].x));
  }
}

// Bits of the largest |x| of eight values; a NaN's if one is.
__device__ __forceinline__ uint32_t max_bits(const float (&x)[8]) {
  auto max3 = [](float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
  };
  return __float_as_uint(max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7])));
}

// The same of eight packed bf16 values.
__device__ __forceinline__ uint32_t max_bits(const uint4 &w) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
  return max(t << 16, t & 0xFFFF0000u);
}

// Codes of this lane's eight channels and the scale byte of its block (four lanes); `m`: the bits of
// its largest magnitude.
__device__ __forceinline__ uint2 quantise8(float (&x)[8], uint32_t m, uint32_t &byte) {
  m = max(m, __shfl_xor_sync(kFullMask, m, 1));
  m = max(m, __shfl_xor_sync(kFullMask, m, 2));
  byte = q8_scale_byte(m);
  if (byte >= kQ8TopByte) {
    if (byte == kQ8NanByte) return make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -240.f * 0x1p120f), 240.f * 0x1p120f);
  }
  const float inv = q8_inv_scale(byte);
  return make_uint2(q8_encode2(x[0], x[1], inv) | (q8_encode2(x[2], x[3], inv) << 16),
                    q8_encode2(x[4], x[5], inv) | (q8_encode2(x[6], x[7], inv) << 16));
}

// kHeads heads a thread, H / kHeads apart, so that the item's coordinates and coefficients serve
// all of them and 3 * kHeads loads are in flight.
template <int D, int kHeads>
__global__ void __launch_bounds__(kAppendThreads, 6) q8_rope_kv_append_kernel(const Q8AppendParams q,
                                                                      uint32_t n_items) {
  const RopeAppendParams &p = q.rope;
  let_successor_start();
  wait_for_predecessor();
  const uint32_t it = blockIdx.x * kAppendThreads + threadIdx.x;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.frames; i += kAppendThreads) {
      const int f = p.frame_idx + i;
      if (debug_check(f >= 0 && p.cap > 0, p.dev_error)) p.slot_frame[f % p.cap] = f;
    }
  Item m;
  // n_items is a multiple of a block's four lanes, so a block's lanes are live together
  const bool live = it < n_items && locate<D, kHeads>(p, it, m);
  if (!live) {
    m.e = m.ce = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) m.cs[u] = make_float2(0.f, 0.f);
  }
  const long long de = static_cast<long long>(p.H / kHeads) * D;
  const long long dce = static_cast<long long>(p.H / kHeads) * p.rows * D;
  uint4 qv[kHeads], kv[kHeads], vv[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    qv[h] = kv[h] = vv[h] = make_uint4(0, 0, 0, 0);
    if (live) {
      qv[h] = ld_plain(static_cast<const __nv_bfloat16 *>(p.q) + m.e + h * de);
      kv[h] = ld_once(static_cast<const __nv_bfloat16 *>(p.k) + m.e + h * de);
      vv[h] = ld_once(static_cast<const __nv_bfloat16 *>(p.v) + m.e + h * de);
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float kx[8], vx[8];
    unpack8(kv[h], kx);
    unpack8(vv[h], vx);
    rotate8(kx, m.cs);
    uint32_t kb, vb;
    const uint2 kc = quantise8(kx, max_bits(kx), kb);
    const uint2 vc = quantise8(vx, max_bits(vv[h]), vb);
    if (!live) continue;
    uint4 qo;
    qo.x = rope_rotate_pair(qv[h].x, m.cs[0]);
    qo.y = rope_rotate_pair(qv[h].y, m.cs[1]);
    qo.z = rope_rotate_pair(qv[h].z, m.cs[2]);
    qo.w = rope_rotate_pair(qv[h].w, m.cs[3]);
    const long long ce = m.ce + h * dce;
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(q.q_out) + m.e + h * de) = qo;
    *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.k_cache) + ce) = kc;
    *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.v_cache) + ce) = vc;
    if ((threadIdx.x & 3) == 0) {
      q.k_scale[ce / kQ8Block] = static_cast<unsigned char>(kb);
      q.v_scale[ce / kQ8Block] = static_cast<unsigned char>(vb);
    }
  }
}

// Eight codes of K and of V a thread and turn, two turns' loads at once: 8 bytes in, 16 out, so
// that a warp's accesses are whole sectors on both sides.
template <int D>
__global__ void __launch_bounds__(kThreads) q8_cache_read_kernel(const Q8ReadParams p) {
  constexpr int kVecs = D / 8, kTurns = 2;
  const long long n = static_cast<long long>(p.n_rows) * kVecs;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  let_successor_start();
  wait_for_predecessor();
  for (long long head = blockIdx.y; head < p.heads; head += gridDim.y) {
    for (long long i0 = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i0 < n;
         i0 += step * kTurns) {
      uint2 w[kTurns][2];
      uint32_t byte[kTurns][2];
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const long long it = i0 + k * step;
        if (it >= n) continue;
        const int r = static_cast<int>(it / kVecs), c = static_cast<int>(it % kVecs);
        const int row = r < p.seg_len[0] ? p.seg_row[0] + r : p.seg_row[1] + (r - p.seg_len[0]);
        const long long src = (head * p.rows + row) * D + c * 8;
        if (!debug_check(head >= 0 && head < p.heads && r >= 0 && r < p.n_rows && row >= 0 &&
                             row < p.rows && c >= 0 && c < kVecs,
                         p.dev_error))
          return;
        if (p.k_out) {
          w[k][0] = *reinterpret_cast<const uint2 *>(p.k_cache + src);
          byte[k][0] = p.k_scale[src / kQ8Block];
        }
        if (p.v_out) {
          w[k][1] = *reinterpret_cast<const uint2 *>(p.v_cache + src);
          byte[k][1] = p.v_scale[src / kQ8Block];
        }
      }
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const long long it = i0 + k * step;
        if (it >= n) continue;
        const long long dst = head * p.n_rows * D + it * 8;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          void *out = t ? p.v_out : p.k_out;
          if (!out) continue;
          const uint32_t m1 = q8_mul1(byte[k][t]), m2 = q8_mul2(byte[k][t]);
          const uint2 a = q8_decode4(w[k][t].x), b = q8_decode4(w[k][t].y);
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + dst) =
              make_uint4(bf16x2_mul(bf16x2_mul(a.x, m1), m2), bf16x2_mul(bf16x2_mul(a.y, m1), m2),
                         bf16x2_mul(bf16x2_mul(b.x, m1), m2), bf16x2_mul(bf16x2_mul(b.y, m1), m2));
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_q8_rope_kv_append(const Q8AppendParams &in, cudaStream_t stream) {
  Q8AppendParams p = in;
  RopeAppendParams &r = p.rope;
  if (r.D != 128 && r.D != 64) return cudaErrorInvalidValue;
  const int heads = r.H % 4 == 0 ? 4 : r.H % 3 == 0 ? 3 : r.H % 2 == 0 ? 2 : 1;
  const long long n_items = static_cast<long long>(r.B) * r.L * (r.H / heads) * (r.D / 8);
  if (n_items < 1 || n_items >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  r.slot0 = r.frame_idx % r.cap;
  r.div_h = make_fastdiv(static_cast<uint32_t>(r.H / heads));
  r.div_l = make_fastdiv(static_cast<uint32_t>(r.L));
  r.div_tf = make_fastdiv(static_cast<uint32_t>(r.Tf));
  r.div_wg = make_fastdiv(static_cast<uint32_t>(r.Wg));
  const unsigned blocks = static_cast<unsigned>((n_items + kAppendThreads - 1) / kAppendThreads);
  const uint32_t n = static_cast<uint32_t>(n_items);
  const bool wide = r.D == 128;
  auto run = [&](auto kernel) {
    return launch_overlapped(kernel, dim3(blocks), kAppendThreads, 0, stream, p, n);
  };
  switch (heads) {
    case 4:
      return run(wide ? q8_rope_kv_append_kernel<128, 4> : q8_rope_kv_append_kernel<64, 4>);
    case 3:
      return run(wide ? q8_rope_kv_append_kernel<128, 3> : q8_rope_kv_append_kernel<64, 3>);
    case 2:
      return run(wide ? q8_rope_kv_append_kernel<128, 2> : q8_rope_kv_append_kernel<64, 2>);
    default:
      return run(wide ? q8_rope_kv_append_kernel<128, 1> : q8_rope_kv_append_kernel<64, 1>);
  }
}

cudaError_t launch_q8_cache_read(const Q8ReadParams &p, cudaStream_t stream) {
  const long long n = static_cast<long long>(p.n_rows) * (p.D / 8);
  const long long bx = (n + 2 * kThreads - 1) / (2 * kThreads);  // two turns a thread
  const dim3 grid(static_cast<unsigned>(bx < (1ll << 30) ? bx : (1ll << 30)),
                  static_cast<unsigned>(p.heads < 65535 ? p.heads : 65535));
  if (p.D != 128 && p.D != 64) return cudaErrorInvalidValue;
  return launch_overlapped(p.D == 128 ? q8_cache_read_kernel<128> : q8_cache_read_kernel<64>, grid,
                           kThreads, 0, stream, p);
}

}  // namespace unstep
