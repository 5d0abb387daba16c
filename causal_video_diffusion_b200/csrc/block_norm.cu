// block_norm.cu -- LayerNorm or RMS norm with affine part and per-frame modulation, alone or after
// the gated residual sum that ends the block before it.
//
// One CTA a row; every pass reads the row again (from L1/L2 after the first).
#include <cuda_bf16.h>

#include "block_norm.h"

namespace unstep {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float ld(const void *p, int type, long long i) {
  return type == UNSTEP_F32 ? static_cast<const float *>(p)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ float row_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

// Mean (0 for RMS) and 1 / sqrt(mean square + eps) of f(c), c < C.
template <class F>
__device__ float2 statistics(const unstep_norm_t &n, int C, F f) {
  float mean = 0.f, s = 0.f;
  if (n.kind == UNSTEP_NORM_LAYER) {
    for (int c = threadIdx.x; c < C; c += kThreads) s += f(c);
    mean = row_sum(s) / C;
  }
  s = 0.f;
  for (int c = threadIdx.x; c < C; c += kThreads) s += (f(c) - mean) * (f(c) - mean);
  return make_float2(mean, 1.f / sqrtf(row_sum(s) / C + n.eps));
}

__device__ __forceinline__ float apply(const unstep_norm_t &n, float2 st, float x, int c,
                                       long long g) {
  float r = (x - st.x) * st.y;
  if (n.weight) r *= ld(n.weight, n.param_type, c);
  if (n.bias) r += ld(n.bias, n.param_type, c);
  if (n.scale) r *= 1.f + ld(n.scale, n.param_type, g * n.mod_stride + c);
  if (n.shift) r += ld(n.shift, n.param_type, g * n.mod_stride + c);
  return r;
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(const NormParams p) {
  extern __shared__ float sum[];  // the row of the new residual (kGated)
  const int C = p.C;
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const long long g = r / p.rows_per_group;
    auto x = [&](int c) { return ld(p.x, p.x_type, r * p.ldx + c); };
    if (kGated) {
      auto y = [&](int c) { return ld(p.y, UNSTEP_BF16, r * p.ldy + c); };
      float2 st = make_float2(0.f, 1.f);
      if (p.has_post) st = statistics(p.post, C, y);
      __syncthreads();
      for (int c = threadIdx.x; c < C; c += kThreads) {
        float v = p.has_post ? apply(p.post, st, y(c), c, g) : y(c);
        if (p.gate) v *= ld(p.gate, p.gate_type, g * p.gate_stride + c);
        v = fmaf(p.res_scale, v, x(c));
        sum[c] = v;
        if (p.x_type == UNSTEP_F32)
          static_cast<float *>(p.x_out)[r * p.ldxo + c] = v;
        else
          static_cast<__nv_bfloat16 *>(p.x_out)[r * p.ldxo + c] = __float2bfloat16_rn(v);
      }
      if (!p.h) continue;
      auto v = [&](int c) { return sum[c]; };
      st = statistics(p.next, C, v);
      for (int c = threadIdx.x; c < C; c += kThreads)
        static_cast<__nv_bfloat16 *>(p.h)[r * p.ldh + c] =
            __float2bfloat16_rn(apply(p.next, st, sum[c], c, g));
    } else {
      const float2 st = statistics(p.next, C, x);
      for (int c = threadIdx.x; c < C; c += kThreads)
        static_cast<__nv_bfloat16 *>(p.h)[r * p.ldh + c] =
            __float2bfloat16_rn(apply(p.next, st, x(c), c, g));
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormParams &p, bool gated, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.rows < (1ll << 30) ? p.rows : (1ll << 30));
  if (gated) {
    const int smem = p.C * static_cast<int>(sizeof(float));
    const cudaError_t e = cudaFuncSetAttribute(
        block_norm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
    if (e != cudaSuccess) return e;
    block_norm_kernel<true><<<grid, kThreads, smem, stream>>>(p);
  } else {
    block_norm_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace unstep
