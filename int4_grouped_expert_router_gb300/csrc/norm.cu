// Norms around a block, fused with its gate, residual scale and residual:
//   b = block * rsqrt(mean(block^2) + eps) * w_post,  h = resid + alpha * g * b,
//   x = h * rsqrt(mean(h^2) + eps) * w_pre.
//
// Bound by memory: every array is read or written once. One CTA takes a row and keeps it in registers
// between the two reductions, which would otherwise cost a second read of the block's output and of h.
// All of a thread's loads are issued before the first reduction. A thread's elements are whole
// 16-byte vectors of memory even where a row does not start at one (an odd D): the arrays share their
// offset from such a boundary, so the row is cut at the boundaries of memory and the first and last
// vector are taken element by element.
//
// Measured: 4096 rows of 6144 (bf16, gated, both norms): 48 us, 5.3 TB/s, 0.78 of a copy's rate; the rest is
// the two reductions, during which a CTA's loads are not replaced by new ones. One row of 6144 (f32): 3.5 us on the
// device, two reductions' latency, less than the call costs on the host.
#include <cuda_bf16.h>

#include <type_traits>

#include "norm.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr float kInf = __builtin_huge_valf();

// Threads of a CTA whose threads hold that many elements of the row (registers).
__host__ __device__ constexpr int max_threads(int held) { return held > 16 ? 544 : 1024; }

// Sum over the CTA; s holds 32 floats per use, and the uses alternate.
__device__ __forceinline__ float block_sum(float v, float* s) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < (int)(blockDim.x >> 5) ? s[lane] : 0.f;
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A vector as it lies in memory: 16 bytes, or one element's bits.
template <int V>
using Raw = std::conditional_t<V == 1, uint32_t, uint4>;

// bf16: the fast exponential is off by about |x| units in the last place, at most 2^-17 where the result is a normal
// number, and h is rounded to 2^-9; the exact exponential and division cost as many instructions as all the rest of the
// kernel. f32: to a few units in the last place over the whole range. e^-|x| = 2^t (1 + r ln 2), t + r the product
// -|x| log2(e) with what its rounding and the factor's lose (4096 gated rows of 6144: 93 us without, 95 us so, 103 us with
// the exact exponential and division).
template <bool BF16>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (BF16) {
    return __fdividef(1.f, 1.f + __expf(-x));
  } else {
    constexpr float kLog2e = 1.4426950408889634074f, kRest = (float)(1.4426950408889634074 - (double)kLog2e), kLn2 = 0.69314718f;
    const float a = fabsf(x) > 128.f ? 128.f : fabsf(x);  // NaN stays
    const float t = -a * kLog2e, r = fmaf(-a, kRest, fmaf(-a, kLog2e, -t));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, r * kLn2, e);
    const float s = __fdividef(1.f, 1.f + e);
    return x < 0.f ? e * s : s;
  }
}

// V consecutive elements from e0 of a row that starts at `row`; those outside 0..D are 0.
template <bool BF16, int V>
__device__ __forceinline__ Raw<V> load_raw(const void* p, size_t row, int e0, int D, bool whole) {
  auto element = [&](int i) -> uint32_t {
    if (e0 + i < 0 || e0 + i >= D) return 0;
    return BF16 ? __ldcg(static_cast<const unsigned short*>(p) + row + e0 + i)
                : __ldcg(static_cast<const uint32_t*>(p) + row + e0 + i);
  };
  if constexpr (V == 1) {
    return element(0);
  } else {
    if (whole) return __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (row + e0) * (BF16 ? 2 : 4)));
    if constexpr (BF16)
      return make_uint4(element(0) | element(1) << 16, element(2) | element(3) << 16, element(4) | element(5) << 16,
                        element(6) | element(7) << 16);
    else
      return make_uint4(element(0), element(1), element(2), element(3));
  }
}

template <bool BF16, int V>
__device__ __forceinline__ void unpack(const Raw<V>& raw, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = __uint_as_float(BF16 ? raw << 16 : raw);
  } else {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (BF16)
        v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      else
        v[i] = __uint_as_float(w[i]);
    }
  }
}

template <bool BF16, int V>
__device__ __forceinline__ void store_vec(void* p, size_t row, int e0, int D, bool whole, const float (&v)[V]) {
  if (whole) {
    if constexpr (BF16 && V == 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&two);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
      return;
    } else if constexpr (!BF16 && V == 4) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + row + e0) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i++) {
    if (e0 + i < 0 || e0 + i >= D) continue;
    if (BF16)
      static_cast<uint16_t*>(p)[row + e0 + i] = f32_to_bf16_rn(v[i]);
    else
      static_cast<float*>(p)[row + e0 + i] = v[i];
  }
}

// A norm's weights: read by every row, so through L1.
template <int V>
__device__ __forceinline__ void load_weight(const float* w, int e0, int D, bool whole, bool aligned, float (&v)[V]) {
  if constexpr (V >= 4) {
    if (whole && aligned) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(w + e0 + i);
        v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; i++) v[i] = e0 + i >= 0 && e0 + i < D ? w[e0 + i] : 0.f;
}

// V elements per vector (16 bytes, or 1 where the arrays do not share their alignment), N vectors per thread.
template <bool BF16, int V, int N>
__global__ void __launch_bounds__(max_threads(N * V), N * V > 16 && N <= 4 ? 2 : 1) norm_kernel(NormArgs a, int shift_step, int* err) {
  constexpr bool kEarly = V > 1 && N <= 4;  // residual and gate wait in registers too
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float s_red[2][32];
  const size_t row = (size_t)blockIdx.x * a.D;
  const int D = a.D;
  // elements by which the row starts after a vector boundary
  const int shift = V == 1 ? 0 : (int)(((uint64_t)blockIdx.x * (uint64_t)D + shift_step) % V);
  const bool w_aligned = shift == 0 && (((uintptr_t)a.w_post | (uintptr_t)a.w_pre) & 15) == 0;
  const bool g_aligned = a.gate_per_row || (shift == 0 && ((uintptr_t)a.gate & 15) == 0);
  float b[N][V];
  Raw<V> raw[N], rs[kEarly ? N : 1], gt[kEarly ? N : 1];
  auto at = [&](int n) { return (n * (int)blockDim.x + (int)threadIdx.x) * V - shift; };
  auto is_whole = [&](int e0) { return e0 >= 0 && e0 + V <= D; };
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e0 = at(n);
    const bool whole = is_whole(e0);
    raw[n] = Raw<V>{};
    if (a.block) raw[n] = load_raw<BF16, V>(a.block, row, e0, D, whole);
    if constexpr (kEarly) {
      if (a.resid) rs[n] = load_raw<BF16, V>(a.resid, row, e0, D, whole);
      if (a.gate) gt[n] = load_raw<BF16, V>(a.gate, a.gate_per_row ? row : 0, e0, D, whole && g_aligned);
    }
  }
  float r = a.alpha;
  if (a.w_post) {
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < N; n++) {
      float t[V];
      unpack<BF16, V>(raw[n], t);
#pragma unroll
      for (int i = 0; i < V; i++) ss = fmaf(t[i], t[i], ss);
    }
    ss = block_sum(ss, s_red[0]);
    if (!(ss < kInf) && threadIdx.x == 0) set_error(err, COLI_E_NONFINITE);
    r = rsqrtf(ss / (float)D + a.eps);
  }
  float hs = 0.f;
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e0 = at(n);
    const bool whole = is_whole(e0);
    float w[V], t[V];
    unpack<BF16, V>(raw[n], b[n]);
    if (a.w_post) {
      load_weight<V>(a.w_post, e0, D, whole, w_aligned, w);
#pragma unroll
      for (int i = 0; i < V; i++) b[n][i] *= r * w[i];
    }
    if (a.gate) {
      if constexpr (!kEarly) gt[0] = load_raw<BF16, V>(a.gate, a.gate_per_row ? row : 0, e0, D, whole && g_aligned);
      unpack<BF16, V>(gt[kEarly ? n : 0], t);
#pragma unroll
      for (int i = 0; i < V; i++) b[n][i] *= a.gate_sigmoid ? sigmoid<BF16>(t[i]) : t[i];
    }
    if (a.resid) {
      if constexpr (!kEarly) rs[0] = load_raw<BF16, V>(a.resid, row, e0, D, whole);
      unpack<BF16, V>(rs[kEarly ? n : 0], t);
#pragma unroll
      for (int i = 0; i < V; i++) b[n][i] = fmaf(a.alpha, b[n][i], t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) b[n][i] *= a.alpha;
    }
#pragma unroll
    for (int i = 0; i < V; i++) hs = fmaf(b[n][i], b[n][i], hs);
  }
  if (a.x || a.h) {
    hs = block_sum(hs, s_red[1]);
    if (!(hs < kInf) && threadIdx.x == 0) set_error(err, COLI_E_NONFINITE);
  }
  r = rsqrtf(hs / (float)D + a.eps);
#pragma unroll
  for (int n = 0; n < N; n++) {
    const int e0 = at(n);
    const bool whole = is_whole(e0);
    if (e0 >= D) break;
    if (a.h) store_vec<BF16, V>(a.h, row, e0, D, whole, b[n]);
    if (a.x) {
      float w[V];
      load_weight<V>(a.w_pre, e0, D, whole, w_aligned, w);
#pragma unroll
      for (int i = 0; i < V; i++) w[i] *= b[n][i] * r;
      store_vec<BF16, V>(a.x, row, e0, D, whole, w);
    }
  }
}

template <bool BF16, int V, int N>
cudaError_t launch_one(coli_ctx* ctx, const NormArgs& a, int threads, int shift_step) {
  return launch_k(norm_kernel<BF16, V, N>, a.S, threads, 0, ctx->stream, true, false, a, shift_step, ctx->d_status);
}

// Vectors per thread. Few rows: as many threads as the row has vectors (one CTA's latency is the call's).
// Many rows: about three vectors each, so that a CTA's barriers stall few warps and several CTAs share an SM.
template <bool BF16, int V>
cudaError_t launch_vec(coli_ctx* ctx, const NormArgs& a, int off) {
  const int vecs = off == 0 && a.D % V == 0 ? a.D / V : (a.D + 2 * (V - 1)) / V;  // at most, whatever the row's shift
  int n = a.S < ctx->num_sms || vecs < 192 ? 1 : vecs < 384 ? 2 : 3;
  while ((vecs + n - 1) / n > max_threads(n * V)) n = n < 4 ? n + 1 : 2 * n;
  const int threads = ((vecs + n - 1) / n + 31) / 32 * 32;
  switch (n) {
    case 1: return launch_one<BF16, V, 1>(ctx, a, threads, off);
    case 2: return launch_one<BF16, V, 2>(ctx, a, threads, off);
    case 3: return launch_one<BF16, V, 3>(ctx, a, threads, off);
    case 4: return launch_one<BF16, V, 4>(ctx, a, threads, off);
    case 8: return launch_one<BF16, V, 8>(ctx, a, threads, off);
  }
  if constexpr (V < 8)
    if (n == 16) return launch_one<BF16, V, 16>(ctx, a, threads, off);
  if constexpr (V == 1) return n == 32 ? launch_one<BF16, V, 32>(ctx, a, threads, off) : launch_one<BF16, V, 64>(ctx, a, threads, off);
  return cudaErrorInvalidValue;  // no row of COLI_MAX_DIM elements comes here
}

}  // namespace

int launch_norm_residual(coli_ctx* ctx, const NormArgs& a) {
  const int elem = a.dtype == COLI_DTYPE_BF16 ? 2 : 4;
  // the arrays that a row indexes share their offset from a 16-byte boundary, or elements are taken one by one
  const void* rows[5] = {a.block, a.resid, a.gate_per_row ? a.gate : nullptr, a.h, a.x};
  int off = -1;
  bool same = true;
  for (const void* p : rows)
    if (p) {
      const int o = (int)((uintptr_t)p & 15);
      same = same && (off < 0 || o == off);
      off = o;
    }
  ProfScope prof(ctx, COLI_KERNEL_NORM);
  cudaError_t e;
  if (a.dtype == COLI_DTYPE_BF16)
    e = same ? launch_vec<true, 8>(ctx, a, off / elem) : launch_vec<true, 1>(ctx, a, 0);
  else
    e = same ? launch_vec<false, 4>(ctx, a, off / elem) : launch_vec<false, 1>(ctx, a, 0);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "norm_residual launch");
  return COLI_OK;
}

}  // namespace coli
