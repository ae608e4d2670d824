// Attention over the 4-bit key/value cache (layout: kv4.h).
//
// For a query row q at position p of its sequence and the visible positions t,
//   x_t = scale sum_g [ s_tg q_g . (n_tg - 8) + o_tg sum(q_g) ],   out = sum_t a_t V_t / sum_t a_t,
// a_t = exp(x_t - max x), one pass over the tokens with a running maximum and sum.
#include "kv4.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kTile = 128;  // tokens per step: one per thread

__device__ __forceinline__ float value_of(uint32_t par, uint32_t n) {
  return __uint_as_float(par & 0xffff0000u) + __uint_as_float(par << 16) * (float)((int)n - 8);
}

// One CTA per (row, query head): a thread scores one token of a tile; then a thread owns channels.
template <bool BF16>
__global__ void __launch_bounds__(kTile) kv4_attn_kernel(Kv4View c, Kv4Plan p, const void* q, long long q_stride,
                                                         int q_heads, float scale, int window, void* out,
                                                         long long out_stride, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float s_q[256], s_a[kTile], s_red[8];
  __shared__ const uint8_t* s_unit[kTile];
  const int row = blockIdx.x / q_heads, qh = blockIdx.x % q_heads, head = qh / (q_heads / c.heads);
  const int tid = threadIdx.x, gs = c.hd / c.ng;
  const int b = kv4_seq_of(p, row);
  int r0, r1;
  kv4_rows(p, b, r0, r1, err);
  if (row < r0 || row >= r1) return;
  const int pos = kv4_len(p, c.page_log2, b, err) - (r1 - row);
  bool finite = true;
  for (int d = tid; d < c.hd; d += kTile) {
    s_q[d] = load_act(q, BF16 ? COLI_DTYPE_BF16 : COLI_DTYPE_F32, (size_t)(row * q_stride + qh * c.hd + d));
    finite = finite && fabsf(s_q[d]) < __int_as_float(0x7f800000);
  }
  if (!finite) set_error(err, COLI_E_NONFINITE);
  __syncthreads();
  float m = -__int_as_float(0x7f800000), l = 0.f, acc[2] = {0.f, 0.f};
  const int first = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
  for (int t0 = first / 16 * 16; t0 <= pos; t0 += kTile) {
    const int t = t0 + tid;
    float x = -__int_as_float(0x7f800000);
    const uint8_t* unit = nullptr;
    if (t >= first && t <= pos) {
      const int page = __ldcg(p.table + (size_t)b * p.table_stride + (t >> c.page_log2));
      if (page < 0 || page >= c.pages) {
        set_error(err, COLI_E_RANGE);
      } else {
        unit = kv4_unit(c, page, head, t & ((1 << c.page_log2) - 1));
        x = 0.f;
        for (int d = 0; d < c.hd; d += 8) {
          const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_k_word(c.hd, t & 15, d / 32, d % 32 / 8)));
          const uint32_t par = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_kscale_at(c.hd) + ((t & 15) * c.ng + d / gs) * 4));
          for (int j = 0; j < 8; j++) x += s_q[d + j] * value_of(par, (w >> (4 * j)) & 15u);
        }
        x *= scale;
      }
    }
    s_unit[tid] = unit;
    float mx = x;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, mx);
    const float base = mn == -__int_as_float(0x7f800000) ? 0.f : mn;
    const float a = expf(x - base);
    s_a[tid] = a;
    float sum = a;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) s_red[4 + (tid >> 5)] = sum;
    __syncthreads();
    const float f = expf(m - base);
    l = l * f + (s_red[4] + s_red[5] + s_red[6] + s_red[7]);
    m = mn;
    for (int h = 0, d = tid; d < c.hd; d += kTile, h++) {
      const int i = d / 32, j = (d % 32) / 16 * 2 + d % 2, r = d % 16 / 2;
      float y = acc[h] * f;
      for (int s = 0; s < kTile && t0 + s <= pos; s++) {
        const uint8_t* un = s_unit[s];
        if (!un) continue;
        const int tt = (t0 + s) & 15;
        const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(un + kv4_v_at(c.hd, c.ng) + kv4_v_word(c.hd, tt >> 1, r, i)));
        const uint32_t par = __ldcg(reinterpret_cast<const uint32_t*>(un + kv4_vscale_at(c.hd, c.ng) + (tt * c.ng + d / gs) * 4));
        y += s_a[s] * value_of(par, (w >> (16 * (tt & 1) + 4 * j)) & 15u);
      }
      acc[h] = y;
    }
    __syncthreads();
  }
  for (int h = 0, d = tid; d < c.hd; d += kTile, h++) {
    const float y = l == 0.f ? 0.f : acc[h] / l;
    const size_t at = (size_t)(row * out_stride + qh * c.hd + d);
    if (BF16)
      static_cast<uint16_t*>(out)[at] = f32_to_bf16_rn(y);
    else
      static_cast<float*>(out)[at] = y;
  }
}

}  // namespace

int launch_kv4_attention(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* q, long long q_stride, int dtype,
                         int q_heads, float scale, int window, void* out, long long out_stride) {
  const long long grid = (long long)p.T * q_heads;
  if (grid > 0x7fffffffll) return fail(ctx, COLI_E_INVAL, "kv4_attention: too many rows for one call");
  ProfScope prof(ctx, COLI_KERNEL_ATTENTION);
  auto kern = dtype == COLI_DTYPE_BF16 ? kv4_attn_kernel<true> : kv4_attn_kernel<false>;
  cudaError_t e = launch_k(kern, (int)grid, kTile, 0, ctx->stream, true, false, c, p, q, q_stride, q_heads, scale, window,
                           out, out_stride, ctx->d_status);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_attention launch");
  return COLI_OK;
}

}  // namespace coli
