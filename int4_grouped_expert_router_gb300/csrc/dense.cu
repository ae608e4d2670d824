// y = resid + act(W x + bias) * mul with 16-bit weights (layout: dense.h).
#include "dense.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ const uint16_t* dense_at(const uint8_t* w, int col_tiles, int o, int i) {
  const uint8_t* tile = w + ((size_t)(o / kDenseRows) * col_tiles + i / kDenseCols) * kDenseTile;
  const int r = o % kDenseRows, chunk = i % kDenseCols / 8;
  return reinterpret_cast<const uint16_t*>(tile + r * 128 + ((chunk ^ (r & 7)) << 4)) + i % 8;
}

__global__ void dense_pack_kernel(const uint16_t* src, int rows, int row0, int O, int I, int col_tiles, uint8_t* w) {
  const long long chunks = (long long)((rows + kDenseRows - 1) / kDenseRows) * kDenseRows * col_tiles * 8;
  for (long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x; n < chunks; n += (long long)gridDim.x * blockDim.x) {
    const int r = (int)(n / (col_tiles * 8)), i0 = (int)(n % (col_tiles * 8)) * 8;
    uint32_t v[4] = {0, 0, 0, 0};
    if (r < rows)
      for (int i = 0; i < 8; i++)
        if (i0 + i < I) v[i / 2] |= (uint32_t)src[(size_t)r * I + i0 + i] << (16 * (i & 1));
    *reinterpret_cast<uint4*>(const_cast<uint16_t*>(dense_at(w, col_tiles, row0 + r, i0))) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

__device__ __forceinline__ float dense_act(float z, int act) {
  switch (act) {
    case COLI_ACT_SILU: return z / (1.f + expf(-z));
    case COLI_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case COLI_ACT_GELU_TANH: return z / (1.f + expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
    case COLI_ACT_RELU: return fmaxf(z, 0.f);
    case COLI_ACT_RELU2: return fmaxf(z, 0.f) * fmaxf(z, 0.f);
  }
  return z;
}

__global__ void dense_kernel(DenseArgs a, int x_dtype, int y_dtype, int col_tiles) {
  griddep_launch_dependents();
  griddep_wait();
  const long long cells = (long long)a.S * a.O;
  for (long long n = (long long)blockIdx.x * blockDim.x + threadIdx.x; n < cells; n += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(n / a.O), o = (int)(n % a.O);
    float z = 0.f;
    for (int i = 0; i < a.I; i++) z = fmaf(bf16_to_f32(*dense_at(a.w, col_tiles, o, i)), load_act(a.x, x_dtype, (size_t)t * a.x_stride + i), z);
    if (!(fabsf(z) < kInf)) set_error(a.err, COLI_E_NONFINITE);
    if (a.bias) z += __ldcg(a.bias + o);
    z = dense_act(z, a.act);
    if (a.mul) z *= load_act(a.mul, y_dtype, (size_t)t * a.mul_stride + o);
    if (a.resid) z += load_act(a.resid, y_dtype, (size_t)t * a.resid_stride + o);
    const size_t to = (size_t)t * a.y_stride + o;
    if (y_dtype == COLI_DTYPE_F32)
      static_cast<float*>(a.y)[to] = z;
    else
      static_cast<uint16_t*>(a.y)[to] = f32_to_bf16_rn(z);
  }
}

}  // namespace

cudaError_t launch_dense_pack(cudaStream_t stream, const uint16_t* src, int rows, int row0, int O, int I, uint8_t* w) {
  dense_pack_kernel<<<1216, 256, 0, stream>>>(src, rows, row0, O, I, (I + kDenseCols - 1) / kDenseCols, w);
  return cudaGetLastError();
}

int launch_dense(coli_ctx* ctx, const DenseArgs& args, int x_dtype, int y_dtype) {
  DenseArgs a = args;
  a.err = ctx->d_status;
  ProfScope prof(ctx, COLI_KERNEL_LINEAR);
  const cudaError_t e = launch_k(dense_kernel, ctx->num_sms * 8, 256, 0, ctx->stream, true, false, a, x_dtype, y_dtype,
                                 (a.I + kDenseCols - 1) / kDenseCols);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "dense_linear launch");
  return COLI_OK;
}

}  // namespace coli
