// Log probabilities of given tokens, entropy and alternatives (logprobs.cu).
#pragma once

#include "coli_internal.h"

namespace coli {

// What a CTA that has read a part of a row leaves: the part's largest entry, the sums s = sum e^(z - b) and t = sum (z - b)
// e^(z - b) (in powers of two) over its base b, and its largest entries in descending order, 0 behind the last.
struct alignas(16) LogprobPart {
  float most, b, s, t;
  uint64_t top[COLI_MAX_TOP];
};

// Rows are shared where there are fewer than kLogprobCtas per SM, by at most as many CTAs as that makes in all.
constexpr int kLogprobCtas = 4;
constexpr int kLogprobMostParts = 64;

// Memory of a context for it: the parts, then an arrival counter per row, zero between calls.
inline size_t logprob_slots(int num_sms) { return (size_t)num_sms * kLogprobCtas; }
inline size_t logprob_bytes(int num_sms) { return logprob_slots(num_sms) * (sizeof(LogprobPart) + sizeof(int)); }

struct LogprobArgs {
  const void* x;
  long long stride;
  int S, V;
  float scale;
  const int32_t* tokens;
  int n;
  float* logp;
  float* entropy;
  int k;
  int32_t* top_id;
  float* top_logp;
  int shift_step;  // elements by which the first row starts after a 16-byte boundary
  int parts, per;  // CTAs of a row, and vectors of each
  LogprobPart* part;
  int* count;
  int* err;
};

int launch_logprobs(coli_ctx* ctx, const LogprobArgs& a, int dtype);

}  // namespace coli
