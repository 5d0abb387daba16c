// window_attn_q8.cu -- windowed attention over the 8-bit KV cache.
//
// One warp for one query row: lane t holds channels t*D/32 .. of q and of the unnormalised output,
// and the warp walks the window's keys with an online softmax (running maximum and sum in fp32).
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "q8.cuh"

namespace unstep {
namespace {

constexpr int kThreads = 256;

template <int D>
__device__ __forceinline__ void load_row(const unsigned char *codes, const unsigned char *scales,
                                         long long row, int lane, float (&x)[D / 32]) {
  constexpr int kPer = D / 32;
  const int ch = lane * kPer;
  const Q8Mul m = q8_mul(scales[row * (D / kQ8Block) + ch / kQ8Block]);
  uint32_t c = 0;
  if (kPer == 4)
    c = *reinterpret_cast<const uint32_t *>(codes + row * D + ch);
  else
    c = *reinterpret_cast<const uint16_t *>(codes + row * D + ch);
  const uint2 d = q8_decode4(c);
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const uint32_t w = bf16x2_mul(bf16x2_mul(i ? d.y : d.x, m.m1), m.m2);
    x[2 * i] = __uint_as_float(w << 16);
    x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) q8_window_attn_kernel(const Q8AttnParams p) {
  constexpr int kPer = D / 32;
  const AttnParams &a = p.attn;
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(a.B) * a.H * a.L;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       w < n; w += step) {
    const int l = static_cast<int>(w % a.L), bh = static_cast<int>(w / a.L);
    const int b = bh / a.H, h = bh - b * a.H;
    const long long at = ((static_cast<long long>(a.b0 + b) * a.L + l) * a.act_H + a.h0 + h) * D +
                         lane * kPer;
    float q[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      q[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at + i]) * a.scale_log2;
      o[i] = 0.f;
    }
    float m = -INFINITY, sum = 0.f;
    for (int s = 0; s < 2; ++s) {
      for (int r = 0; r < a.seg_len[s]; ++r) {
        const long long row = static_cast<long long>(bh) * a.rows + a.seg_row[s] + r;
        float x[kPer];
        load_row<D>(p.k_cache, p.k_scale, row, lane, x);
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) t = fmaf(q[i], x[i], t);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
        const float mn = fmaxf(m, t), f = exp2f(m - mn), e = exp2f(t - mn);
        load_row<D>(p.v_cache, p.v_scale, row, lane, x);
        m = mn;
        sum = fmaf(sum, f, e);
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = fmaf(o[i], f, e * x[i]);
      }
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      static_cast<__nv_bfloat16 *>(a.out)[at + i] = __float2bfloat16_rn(o[i] * inv);
  }
}

}  // namespace

cudaError_t launch_q8_window_attn(int D, const Q8AttnParams &p, cudaStream_t stream) {
  const long long n = static_cast<long long>(p.attn.B) * p.attn.H * p.attn.L;
  const long long blocks = (n + kThreads / 32 - 1) / (kThreads / 32);
  const unsigned grid = static_cast<unsigned>(blocks < (1ll << 30) ? blocks : (1ll << 30));
  if (D == 128)
    q8_window_attn_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else if (D == 64)
    q8_window_attn_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace unstep
