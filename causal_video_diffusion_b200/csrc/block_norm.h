// block_norm.h -- launch parameters of the norms before and after a DiT block.
#pragma once

#include <cuda_runtime.h>

#include "../../include/unstep.h"
#include "internal.h"

namespace unstep {

struct NormParams {
  const void *x;       // bf16 or fp32 rows
  const void *y;       // bf16 rows of the block's output (gate form), else NULL
  const void *gate;    // or NULL: 1
  void *x_out;         // the new residual rows (gate form)
  void *h;             // bf16 normed rows, or NULL (gate form without a next norm)
  long long ldx, ldy, ldxo, ldh, gate_stride;
  long long rows, rows_per_group;
  int C;
  int x_type, gate_type;
  int has_post;
  float res_scale;
  unstep_norm_t post, next;
  // set by launch_block_norm: rows and groups below 2^31, division by rows_per_group, every fp32
  // pointer on 32 bytes (row and group strides are multiples of 8 elements)
  bool narrow, wide;
  FastDiv div_group;
  long long sets, extra;  // sets of rows a CTA takes; the first `extra` CTAs take one more
};

// gated = false: h = next(x).  gated = true: x_out = x + res_scale * gate * post(y), h = next of it.
cudaError_t launch_block_norm(const NormParams &p, bool gated, cudaStream_t stream);

}  // namespace unstep
