// Norms around a block, fused with its gate, residual scale and residual:
//   b = block * rsqrt(mean(block^2) + eps) * w_post,  h = resid + alpha * g * b,
//   x = h * rsqrt(mean(h^2) + eps) * w_pre.
#include "norm.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* s) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kThreads / 32; i++) t += s[i];
  return t;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs a, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float s_red[kThreads / 32];
  extern __shared__ float s_h[];
  const size_t at = (size_t)blockIdx.x * a.D;
  float r = 1.f;
  if (a.w_post) {
    float ss = 0.f;
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      const float b = load_act(a.block, a.dtype, at + d);
      ss += b * b;
    }
    ss = block_sum(ss, s_red);
    if (!(ss < __int_as_float(0x7f800000)) && threadIdx.x == 0) set_error(err, COLI_E_NONFINITE);
    r = rsqrtf(ss / (float)a.D + a.eps);
  }
  float hs = 0.f;
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float h = a.resid ? load_act(a.resid, a.dtype, at + d) : 0.f;
    if (a.block) {
      float b = load_act(a.block, a.dtype, at + d);
      if (a.w_post) b *= r * a.w_post[d];
      if (a.gate) {
        const float g = load_act(a.gate, a.dtype, (a.gate_per_row ? at : 0) + d);
        b *= a.gate_sigmoid ? 1.f / (1.f + expf(-g)) : g;
      }
      h += a.alpha * b;
    }
    s_h[d] = h;
    hs += h * h;
  }
  hs = block_sum(hs, s_red);
  if (!(hs < __int_as_float(0x7f800000)) && threadIdx.x == 0) set_error(err, COLI_E_NONFINITE);
  r = rsqrtf(hs / (float)a.D + a.eps);
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    const float h = s_h[d];
    const float x = a.x ? h * r * a.w_pre[d] : 0.f;
    if (a.dtype == COLI_DTYPE_BF16) {
      if (a.h) static_cast<uint16_t*>(a.h)[at + d] = f32_to_bf16_rn(h);
      if (a.x) static_cast<uint16_t*>(a.x)[at + d] = f32_to_bf16_rn(x);
    } else {
      if (a.h) static_cast<float*>(a.h)[at + d] = h;
      if (a.x) static_cast<float*>(a.x)[at + d] = x;
    }
  }
}

}  // namespace

int launch_norm_residual(coli_ctx* ctx, const NormArgs& a) {
  const size_t smem = (size_t)a.D * 4;
  cudaError_t e = cudaFuncSetAttribute(norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, COLI_MAX_DIM * 4);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "norm_residual attribute");
  ProfScope prof(ctx, COLI_KERNEL_NORM);
  e = launch_k(norm_kernel, a.S, kThreads, smem, ctx->stream, true, false, a, ctx->d_status);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "norm_residual launch");
  return COLI_OK;
}

}  // namespace coli
