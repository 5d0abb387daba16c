// block_norm.cu -- LayerNorm or RMS norm with affine part and per-frame modulation, alone or after
// the gated residual sum that ends the block before it.
//
// A row lives in registers, spread over as many threads as hold one vector of 8 channels each (two
// above 2048 channels, four above 8192): up to 256 channels part of a warp or a warp, behind that
// whole warps.  Every statistic is taken from registers (the variance around the mean, in a second
// pass) and each byte of x, y, x_out and h moves once.  The grid is persistent; a row's data are
// loaded while the row before it is worked on.  Long chunks are bound by HBM and by issue slots (the
// sums and addresses of so few channels a thread): the gated form moves 5.2 TB/s for 65536 rows of
// 1536 channels, the norm alone 3.6 TB/s.  A whole row a warp costs fewer instructions, but its
// serial chain of loads, sums and parameters is not hidden by the few warps that then fit: 4680
// gated fp32 rows of 1536 take 47 us from a cold L2, 25 us this way.
#include <cuda_bf16.h>

#include "block_norm.h"

namespace unstep {
namespace {

constexpr uint32_t kFullMask = 0xFFFFFFFFu;
constexpr int kSms = 148;

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight fp32 values: one 32-byte access where the launch's fp32 pointers allow it (a lane's two
// 16-byte ones use half of every sector they touch).
__device__ __forceinline__ void load_f32(const float *s, bool wide, float (&x)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                   "=f"(x[6]), "=f"(x[7])
                 : "l"(s)
                 : "memory");
  } else {
    const float4 a = reinterpret_cast<const float4 *>(s)[0];
    const float4 b = reinterpret_cast<const float4 *>(s)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

__device__ __forceinline__ void store_f32(float *d, bool wide, const float (&x)[8]) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4 *>(d)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(d)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Eight parameters of either type (the same for the whole launch).
__device__ __forceinline__ void param8(const void *p, int type, bool wide, long long at,
                                       float (&x)[8]) {
  if (type == UNSTEP_F32)
    load_f32(static_cast<const float *>(p) + at, wide, x);
  else
    unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at), x);
}

// Vector v of this thread is channels 8 (first + v * kStep) .. of its row.
template <int kLanes, int kVecs, int kWarps>
struct Row {
  static constexpr int kStep = kLanes * kWarps;
  using Values = float[kVecs][8];
  int first, vecs;           // vecs = C / 8
  float inv_c;
  bool wide;
  float (*part)[kWarps];     // the warps' partial sums, one line for each sum of a row

  __device__ __forceinline__ bool in(int v) const { return first + v * kStep < vecs; }
  __device__ __forceinline__ int channel(int v) const { return 8 * (first + v * kStep); }

  __device__ __forceinline__ float sum(float s, int line) const {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(kFullMask, s, d);
    if constexpr (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) part[line][threadIdx.x >> 5] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += part[line][w];
    }
    return s;
  }

  // x -> norm(x), affine and modulated; lines `line` and `line + 1` of part.
  __device__ __forceinline__ void norm(const unstep_norm_t &n, long long group, Values &x,
                                       int line) const {
    if (n.kind == UNSTEP_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[v][i];  // zeros behind the row's end
      const float mean = sum(s, line) * inv_c;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(x[v][i], x[v][i], q);
      if (in(v)) s += q;
    }
    const float rstd = rsqrtf(fmaf(sum(s, line + 1), inv_c, n.eps));
    const long long mod = group * n.mod_stride;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!in(v)) continue;
      const int c = channel(v);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] *= rstd;
      if (n.weight) {
        param8(n.weight, n.param_type, wide, c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] *= q[i];
      }
      if (n.bias) {
        param8(n.bias, n.param_type, wide, c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] += q[i];
      }
      if (n.scale) {
        param8(n.scale, n.param_type, wide, mod + c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] = fmaf(x[v][i], q[i], x[v][i]);
      }
      if (n.shift) {
        param8(n.shift, n.param_type, wide, mod + c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] += q[i];
      }
    }
  }
};

template <int kWarps>
constexpr int threads_of() {
  return kWarps > 1 ? 32 * kWarps : 128;
}

// CTAs of an SM: registers for the row, the next row and y beside it.
template <int kVecs, int kWarps, bool kF32, bool kGated>
constexpr int ctas_of() {
  constexpr int regs = 44 + kVecs * (8 + (kF32 ? 8 : 4) + (kGated ? 12 : 0));
  constexpr int n = 65536 / threads_of<kWarps>() / ((regs + 7) / 8 * 8);
  return n < 1 ? 1 : (n > 2048 / threads_of<kWarps>() ? 2048 / threads_of<kWarps>() : n);
}

template <int kLanes, int kVecs, int kWarps, bool kF32, bool kGated>
__global__ void __launch_bounds__(threads_of<kWarps>(), (ctas_of<kVecs, kWarps, kF32, kGated>()))
    block_norm_kernel(const NormParams p) {
  constexpr int kRows = threads_of<kWarps>() / (kLanes * kWarps);  // rows of a CTA at once
  __shared__ float part[kWarps > 1 ? 8 : 1][kWarps];
  Row<kLanes, kVecs, kWarps> row;
  row.first = threadIdx.x % (kLanes * kWarps);
  row.vecs = p.C / 8;
  row.inv_c = 1.f / static_cast<float>(p.C);
  row.wide = p.wide;
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  long long r = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / (kLanes * kWarps);
  float xn[kVecs][kF32 ? 8 : 1];       // the next row, as loaded
  uint4 xw[kVecs], yw[kVecs];
  auto fetch = [&](long long at) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (at >= p.rows || !row.in(v)) continue;
      const int c = row.channel(v);
      if constexpr (kF32)
        load_f32(static_cast<const float *>(p.x) + at * p.ldx + c, p.wide, xn[v]);
      else
        xw[v] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) +
                                                 at * p.ldx + c);
      if constexpr (kGated)
        yw[v] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.y) +
                                                 at * p.ldy + c);
    }
  };
  fetch(r);
  // a CTA's threads take the same number of turns: rows behind the last are zeros, unstored
  long long base = static_cast<long long>(blockIdx.x) * kRows;
  for (int turn = 0; base < p.rows; base += step, r += step, turn ^= 4) {
    // the sums' lines alternate: a warp may still read this turn's when another starts the next
    row.part = part + (kWarps > 1 ? turn : 0);
    const bool live = r < p.rows;
    const long long g = p.narrow ? static_cast<long long>(fdiv(static_cast<uint32_t>(r), p.div_group))
                                 : r / p.rows_per_group;
    float x[kVecs][8];
    float y[kGated ? kVecs : 1][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const bool on = live && row.in(v);
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] = on ? xn[v][i] : 0.f;
      } else {
        unpack8(on ? xw[v] : make_uint4(0, 0, 0, 0), x[v]);
      }
      if constexpr (kGated) unpack8(on ? yw[v] : make_uint4(0, 0, 0, 0), y[v]);
    }
    fetch(r + step);
    if constexpr (kGated) {
      if (p.has_post) row.norm(p.post, live ? g : 0, y, 0);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!live || !row.in(v)) continue;
        const int c = row.channel(v);
        if (p.gate) {
          float q[8];
          param8(p.gate, p.gate_type, p.wide, g * p.gate_stride + c, q);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] *= q[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] = fmaf(p.res_scale, y[v][i], x[v][i]);
        if constexpr (kF32)
          store_f32(static_cast<float *>(p.x_out) + r * p.ldxo + c, p.wide, x[v]);
        else
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.x_out) + r * p.ldxo + c) =
              pack8(x[v]);
      }
      if (!p.h) continue;
    }
    row.norm(p.next, live ? g : 0, x, kGated ? 2 : 0);
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (live && row.in(v))
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.h) + r * p.ldh +
                                   row.channel(v)) = pack8(x[v]);
  }
}

template <int kLanes, int kVecs, int kWarps, bool kF32, bool kGated>
void start(const NormParams &p, cudaStream_t stream) {
  constexpr int kThreads = threads_of<kWarps>(), kRows = kThreads / (kLanes * kWarps);
  constexpr long long kMost = static_cast<long long>(kSms) * ctas_of<kVecs, kWarps, kF32, kGated>();
  const long long blocks = (p.rows + kRows - 1) / kRows;
  block_norm_kernel<kLanes, kVecs, kWarps, kF32, kGated>
      <<<static_cast<unsigned>(blocks < kMost ? blocks : kMost), kThreads, 0, stream>>>(p);
}

template <int kLanes, int kVecs, int kWarps>
cudaError_t launch(const NormParams &p, bool gated, cudaStream_t stream) {
  const bool f32 = p.x_type == UNSTEP_F32;
  if (gated && f32)
    start<kLanes, kVecs, kWarps, true, true>(p, stream);
  else if (gated)
    start<kLanes, kVecs, kWarps, false, true>(p, stream);
  else if (f32)
    start<kLanes, kVecs, kWarps, true, false>(p, stream);
  else
    start<kLanes, kVecs, kWarps, false, false>(p, stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const NormParams &in, bool gated, cudaStream_t s) {
  NormParams p = in;
  p.narrow = p.rows < (1ll << 31) && p.rows_per_group < (1ll << 31);
  if (p.narrow) p.div_group = make_fastdiv(static_cast<uint32_t>(p.rows_per_group));
  uintptr_t low = 0;  // fp32 pointers' low bits
  auto add = [&](const void *q, int type) {
    if (type == UNSTEP_F32) low |= reinterpret_cast<uintptr_t>(q);
  };
  auto add_norm = [&](const unstep_norm_t &n) {
    add(n.weight, n.param_type), add(n.bias, n.param_type);
    add(n.scale, n.param_type), add(n.shift, n.param_type);
  };
  add(p.x, p.x_type), add(p.x_out, p.x_type), add(p.gate, p.gate_type);
  if (p.has_post) add_norm(p.post);
  add_norm(p.next);
  p.wide = (low & 31) == 0;
  if (p.C <= 64) return launch<8, 1, 1>(p, gated, s);
  if (p.C <= 128) return launch<16, 1, 1>(p, gated, s);
  if (p.C <= 256) return launch<32, 1, 1>(p, gated, s);
  if (p.C <= 512) return launch<32, 1, 2>(p, gated, s);
  if (p.C <= 1024) return launch<32, 1, 4>(p, gated, s);
  if (p.C <= 1536) return launch<32, 1, 6>(p, gated, s);
  if (p.C <= 2048) return launch<32, 1, 8>(p, gated, s);
  if (p.C <= 4096) return launch<32, 2, 8>(p, gated, s);
  if (p.C <= 8192) return launch<32, 2, 16>(p, gated, s);
  return launch<32, 4, 16>(p, gated, s);
}

}  // namespace unstep
