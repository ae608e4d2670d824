// Norms around a block fused with its gate, residual scale and residual (norm.cu).
#pragma once

#include "coli_internal.h"

namespace coli {

struct NormArgs {
  const void* block;
  const void* resid;
  const void* gate;
  bool gate_per_row;  // gate is [S x D]; otherwise [D]
  bool gate_sigmoid;
  float alpha;
  const float* w_post;
  const float* w_pre;
  float eps;
  int dtype, S, D;
  void* h;
  void* x;
};

int launch_norm_residual(coli_ctx* ctx, const NormArgs& a);

}  // namespace coli
