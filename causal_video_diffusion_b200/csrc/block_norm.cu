// block_norm.cu -- LayerNorm or RMS norm with affine part and per-frame modulation, alone or after
// the gated residual sum that ends the block before it.
//
// A row lives in registers, spread over as many threads as hold one vector of 8 channels each (two
// above 2048 channels, four above 8192): up to 256 channels part of a warp or a warp, behind that
// whole warps.  Every statistic is taken from registers (the variance around the mean, in a second
// pass) and each byte of x, y, x_out and h moves once.  The grid is persistent, a CTA takes
// consecutive rows, and a row is loaded while the one before it is worked on; what all rows of a
// group share (weight, bias, modulation, gate) is folded into one factor and one term a channel and
// stays in registers until the group changes.  What bounds it is HBM for long gated chunks (30000
// fp32 rows of 1536 channels: 89 us, 6.2 TB/s), and the chain of loads and two sums a row, which only
// many resident CTAs hide, for the norm alone (65536 rows of 1536: 81 us, 5.0 TB/s) and for ordinary
// chunks (4680 rows of 1536, call after call: 16.9 us gated, 7.9 us the norm).  Measured instead for
// the gated 4680 rows, 18.7 us before launches overlapped: parameters read for every row 22 us, two
// vectors a thread 22-24, a row a warp 29, two to four rows loaded ahead 25-28 (fewer CTAs fit).  Above
// 8192 channels the gated form's parameters spill (1.7 to 2.2 TB/s).
#include <cuda_bf16.h>

#include "block_norm.h"
#include "internal.h"
#include "sm100.cuh"

namespace unstep {
namespace {

constexpr uint32_t kFullMask = 0xFFFFFFFFu;
constexpr int kSms = 148;

// Eight channels as four packed pairs (low, high) of fp32.
struct Oct {
  uint64_t p[4];
};

__device__ __forceinline__ uint64_t both(float x) { return f2_make(x, x); }

__device__ __forceinline__ Oct zeros() { return Oct{{0, 0, 0, 0}}; }

__device__ __forceinline__ Oct unpack8(const uint4 &w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.p[i] = f2_make(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  return o;
}

__device__ __forceinline__ uint4 pack8(const Oct &o) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_split(o.p[i], lo, hi);
    u[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight fp32 values: one 32-byte access where the launch's fp32 pointers allow it (a lane's two
// 16-byte ones use half of every sector they touch).
__device__ __forceinline__ Oct load_f32(const float *s, bool wide) {
  Oct o;
  if (wide) {
    asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                 : "=l"(o.p[0]), "=l"(o.p[1]), "=l"(o.p[2]), "=l"(o.p[3])
                 : "l"(s)
                 : "memory");
  } else {
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(s)[0];
    const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(s)[1];
    o = Oct{{a.x, a.y, b.x, b.y}};
  }
  return o;
}

__device__ __forceinline__ void store_f32(float *d, bool wide, const Oct &o) {
  if (wide) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(d), "l"(o.p[0]), "l"(o.p[1]),
                 "l"(o.p[2]), "l"(o.p[3])
                 : "memory");
  } else {
    reinterpret_cast<ulonglong2 *>(d)[0] = make_ulonglong2(o.p[0], o.p[1]);
    reinterpret_cast<ulonglong2 *>(d)[1] = make_ulonglong2(o.p[2], o.p[3]);
  }
}

// Eight parameters of either type (the same for the whole launch).
__device__ __forceinline__ Oct param8(const void *p, int type, bool wide, long long at) {
  if (type == UNSTEP_F32) return load_f32(static_cast<const float *>(p) + at, wide);
  return unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at));
}

// Vector v of this thread is channels 8 (first + v * kStep) .. of its row.
template <int kLanes, int kVecs, int kWarps>
struct Row {
  static constexpr int kStep = kLanes * kWarps;
  static constexpr int kLine = (kWarps + 3) / 4 * 4;
  int first, vecs;           // vecs = C / 8
  float inv_c;
  bool wide;
  float (*part)[kLine];      // the warps' partial sums, one line for each sum of a row

  __device__ __forceinline__ bool in(int v) const { return first + v * kStep < vecs; }
  __device__ __forceinline__ int channel(int v) const { return 8 * (first + v * kStep); }

  __device__ __forceinline__ float sum(uint64_t s2, int line) const {
    float lo, hi;
    f2_split(s2, lo, hi);
    float s = lo + hi;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(kFullMask, s, d);
    if constexpr (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) part[line][threadIdx.x >> 5] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int w = 0; w < kLine; w += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(&part[line][w]);
        s += q.x;
        if (w + 1 < kWarps) s += q.y;
        if (w + 2 < kWarps) s += q.z;
        if (w + 3 < kWarps) s += q.w;
      }
    }
    return s;
  }

  // x -> (x - mean) / sqrt(variance + eps) (RMS: mean 0) as x and the factor that is returned;
  // lines `line` and `line + 1` of part.
  __device__ __forceinline__ float normalise(const unstep_norm_t &n, Oct (&x)[kVecs],
                                             int line) const {
    if (n.kind == UNSTEP_NORM_LAYER) {
      uint64_t s = 0;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fadd2(s, x[v].p[i]);  // zeros behind the row's end
      const uint64_t shift = both(-sum(s, line) * inv_c);
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v].p[i] = fadd2(x[v].p[i], shift);
    }
    uint64_t s = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      uint64_t q = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) q = ffma2(x[v].p[i], x[v].p[i], q);
      if (in(v)) s = fadd2(s, q);
    }
    return rsqrtf(fmaf(sum(s, line + 1), inv_c, n.eps));
  }

  // A norm's affine part and modulation for a group, as one factor and one term a channel:
  // (n * weight + bias) * (1 + scale) + shift = n * a + c.
  __device__ __forceinline__ void parameters(const unstep_norm_t &n, long long group,
                                             Oct (&a)[kVecs], Oct (&c)[kVecs]) const {
    const long long mod = group * n.mod_stride;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int ch = channel(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[v].p[i] = both(1.f);
      c[v] = zeros();
      if (!in(v)) continue;
      if (n.weight) a[v] = param8(n.weight, n.param_type, wide, ch);
      if (n.bias) c[v] = param8(n.bias, n.param_type, wide, ch);
      if (n.scale) {
        const Oct q = param8(n.scale, n.param_type, wide, mod + ch);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[v].p[i] = ffma2(a[v].p[i], q.p[i], a[v].p[i]);
          c[v].p[i] = ffma2(c[v].p[i], q.p[i], c[v].p[i]);
        }
      }
      if (n.shift) {
        const Oct q = param8(n.shift, n.param_type, wide, mod + ch);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[v].p[i] = fadd2(c[v].p[i], q.p[i]);
      }
    }
  }
};

template <int kWarps>
constexpr int threads_of() {
  return kWarps > 1 ? 32 * kWarps : 128;
}

enum Mode { kNorm, kGated, kGatedPost };  // h = next(x); with the residual sum; and post(y) in it

// CTAs of an SM: registers for the row, the next row, y beside them, and the parameters.
template <int kVecs, int kWarps, bool kF32, Mode kMode>
constexpr int ctas_of() {
  constexpr int regs = 24 + kVecs * ((kF32 ? 16 : 12) + 16 + (kMode == kNorm ? 0 : 20) +
                                     (kMode == kGatedPost ? 8 : 0));
  constexpr int n = 65536 / threads_of<kWarps>() / ((regs + 7) / 8 * 8);
  return n < 1 ? 1 : (n > 2048 / threads_of<kWarps>() ? 2048 / threads_of<kWarps>() : n);
}

template <int kLanes, int kVecs, int kWarps, bool kF32, Mode kMode>
__global__ void __launch_bounds__(threads_of<kWarps>(), (ctas_of<kVecs, kWarps, kF32, kMode>()))
    block_norm_kernel(const NormParams p) {
  constexpr int kRows = threads_of<kWarps>() / (kLanes * kWarps);  // rows of a CTA at once
  using Place = Row<kLanes, kVecs, kWarps>;
  __shared__ __align__(16) float part[kWarps > 1 ? 8 : 1][Place::kLine];
  Place row;
  row.first = threadIdx.x % (kLanes * kWarps);
  row.vecs = p.C / 8;
  row.inv_c = 1.f / static_cast<float>(p.C);
  row.wide = p.wide;
  // this CTA's turns: consecutive sets of kRows rows, so that the group seldom changes
  const long long b = blockIdx.x;
  const long long set0 = b * p.sets + (b < p.extra ? b : p.extra);
  const long long set1 = set0 + p.sets + (b < p.extra ? 1 : 0);
  long long r = set0 * kRows + threadIdx.x / (kLanes * kWarps);
  let_successor_start();
  wait_for_predecessor();
  // this thread's vector 0 in row r of each tensor
  constexpr int kX = kF32 ? 4 : 2;
  const char *px = static_cast<const char *>(p.x) + (r * p.ldx + row.channel(0)) * kX;
  const char *py = nullptr;
  char *po = nullptr;
  if constexpr (kMode != kNorm) {
    py = static_cast<const char *>(p.y) + (r * p.ldy + row.channel(0)) * 2;
    po = static_cast<char *>(p.x_out) + (r * p.ldxo + row.channel(0)) * kX;
  }
  char *ph = static_cast<char *>(p.h) + (r * p.ldh + row.channel(0)) * 2;
  // the next row as loaded; behind a row's end and behind the last row whatever was there before,
  // zeros to begin with (no sum of a row that is stored takes it in)
  Oct xn[kF32 ? kVecs : 1];
  uint4 xw[kVecs], yw[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    if constexpr (kF32) xn[v] = zeros();
    xw[v] = yw[v] = make_uint4(0, 0, 0, 0);
  }
  auto fetch = [&] {
    constexpr int kStride = 8 * Place::kStep;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!row.in(v)) continue;
      if constexpr (kF32)
        xn[v] = load_f32(reinterpret_cast<const float *>(px) + v * kStride, p.wide);
      else
        xw[v] = *reinterpret_cast<const uint4 *>(px + v * kStride * 2);
      if constexpr (kMode != kNorm) yw[v] = *reinterpret_cast<const uint4 *>(py + v * kStride * 2);
    }
  };
  if (r < p.rows) fetch();
  // the group's parameters: h = n(x) * a + c, x_out = x + n(y) * ga + gc
  Oct a[kVecs], c[kVecs], ga[kVecs], gc[kVecs];
  long long group = -1;
  for (long long set = set0; set < set1; ++set) {
    // the sums' lines alternate: a warp may still read this turn's when another starts the next
    if constexpr (kWarps > 1) row.part = part + (set & 1) * 4;
    const bool live = r < p.rows;
    const long long g =
        !live ? 0 : p.narrow ? static_cast<long long>(fdiv(static_cast<uint32_t>(r), p.div_group))
                             : r / p.rows_per_group;
    if (g != group) {
      group = g;
      if (p.h) row.parameters(p.next, g, a, c);
      if constexpr (kMode != kNorm) {
        if constexpr (kMode == kGatedPost) row.parameters(p.post, g, ga, gc);
        const uint64_t res = both(p.res_scale);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          Oct q;
#pragma unroll
          for (int i = 0; i < 4; ++i) q.p[i] = res;
          if (p.gate && row.in(v)) {
            q = param8(p.gate, p.gate_type, p.wide, g * p.gate_stride + row.channel(v));
#pragma unroll
            for (int i = 0; i < 4; ++i) q.p[i] = fmul2(q.p[i], res);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ga[v].p[i] = kMode == kGatedPost ? fmul2(ga[v].p[i], q.p[i]) : q.p[i];
            if constexpr (kMode == kGatedPost) gc[v].p[i] = fmul2(gc[v].p[i], q.p[i]);
          }
        }
      }
    }
    Oct x[kVecs], y[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if constexpr (kF32)
        x[v] = xn[v];
      else
        x[v] = unpack8(xw[v]);
      if constexpr (kMode != kNorm) y[v] = unpack8(yw[v]);
    }
    r += kRows;
    px += kRows * p.ldx * kX;
    if constexpr (kMode != kNorm) py += kRows * p.ldy * 2;
    if (r < p.rows && set + 1 < set1) fetch();
    if constexpr (kMode != kNorm) {
      uint64_t rstd = both(1.f);
      if constexpr (kMode == kGatedPost) rstd = both(row.normalise(p.post, y, 0));
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!row.in(v)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kMode == kGatedPost) {
            x[v].p[i] = fadd2(x[v].p[i], ffma2(y[v].p[i], fmul2(rstd, ga[v].p[i]), gc[v].p[i]));
          } else {
            x[v].p[i] = ffma2(y[v].p[i], ga[v].p[i], x[v].p[i]);
          }
        }
        if (!live) continue;
        if constexpr (kF32)
          store_f32(reinterpret_cast<float *>(po) + v * 8 * Place::kStep, p.wide, x[v]);
        else
          *reinterpret_cast<uint4 *>(po + v * 16 * Place::kStep) = pack8(x[v]);
      }
      po += kRows * p.ldxo * kX;
      if (!p.h) continue;
    }
    const uint64_t rstd = both(row.normalise(p.next, x, kMode == kNorm ? 0 : 2));
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!live || !row.in(v)) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[v].p[i] = ffma2(x[v].p[i], fmul2(rstd, a[v].p[i]), c[v].p[i]);
      *reinterpret_cast<uint4 *>(ph + v * 16 * Place::kStep) = pack8(x[v]);
    }
    ph += kRows * p.ldh * 2;
  }
}

template <int kLanes, int kVecs, int kWarps, bool kF32, Mode kMode>
cudaError_t start(const NormParams &in, cudaStream_t stream) {
  constexpr int kThreads = threads_of<kWarps>(), kRows = kThreads / (kLanes * kWarps);
  constexpr long long kMost = static_cast<long long>(kSms) * ctas_of<kVecs, kWarps, kF32, kMode>();
  NormParams p = in;
  const long long sets = (p.rows + kRows - 1) / kRows, grid = sets < kMost ? sets : kMost;
  p.sets = sets / grid;
  p.extra = sets % grid;
  return launch_overlapped(block_norm_kernel<kLanes, kVecs, kWarps, kF32, kMode>,
                           dim3(static_cast<unsigned>(grid)), kThreads, 0, stream, p);
}

template <int kLanes, int kVecs, int kWarps>
cudaError_t launch(const NormParams &p, bool gated, cudaStream_t stream) {
  const bool f32 = p.x_type == UNSTEP_F32;
  if (!gated)
    return f32 ? start<kLanes, kVecs, kWarps, true, kNorm>(p, stream)
               : start<kLanes, kVecs, kWarps, false, kNorm>(p, stream);
  if (!p.has_post)
    return f32 ? start<kLanes, kVecs, kWarps, true, kGated>(p, stream)
               : start<kLanes, kVecs, kWarps, false, kGated>(p, stream);
  return f32 ? start<kLanes, kVecs, kWarps, true, kGatedPost>(p, stream)
             : start<kLanes, kVecs, kWarps, false, kGatedPost>(p, stream);
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
  // The narrowest place that holds a row's vectors: lanes of a warp, then warps, one vector a
  // thread as long as that keeps several CTAs on an SM, more above.  Threads behind the row's end
  // only pass the barriers, so a step too wide costs its share of the resident rows.  TB/s of the
  // norm of bf16 rows and of gated fp32 rows (46 million elements), with the step and with the next
  // one above in its place: 128 channels 4.98 and 6.04 against 3.01 and 4.79; 512: 4.89 and 6.16,
  // 2.65 and 4.89; 1536: 4.64 and 6.23, 3.61 and 5.65; 1280, inside that step: 3.94 and 5.86, 3.10
  // and 5.20.  One vector or two a thread: 4096 channels 5.02 and 6.01 with two in 8 warps, 3.98
  // and 5.30 with one in 16; 2048: 4.44 and 6.23 with one in 8, 5.12 and 5.94 with two in 4.  Two
  // or four: 8192 channels 4.10 and 5.92 with two in 16, 3.78 and 5.48 with four in 8.  Widths that
  // lie badly: 2560 runs at 4.11 and 5.49, 5120 at 3.22 and 5.36, 6144 at 3.60 and 5.81.
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
