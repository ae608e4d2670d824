// Rotary positions (rotary.cu).
#pragma once

#include "coli_internal.h"

namespace coli {

struct RotarySide {  // q or k: rows of heads x head_dim, strides in elements
  const void* in;
  void* out;
  long long in_stride, out_stride;
  int heads;
};

struct RotaryArgs {
  RotarySide side[2];
  int hd, rot;
  const uint64_t* freqs;  // turns per position, 64-bit fractions
  float scale;
  int T;
  const int32_t* positions;  // or the plan:
  const int32_t* q_start;
  const int32_t* lens;
  int B;
  int* err;
};

int rotary_freqs(int rot, double base, int scaling, double factor, double original, double low, double high, uint64_t* out);
int launch_rotary(coli_ctx* ctx, const RotaryArgs& a, int dtype, bool interleaved);

}  // namespace coli
