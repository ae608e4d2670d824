// Writing tokens into the 4-bit key/value cache and reading them back (layout: kv4.h).
#include "kv4.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, long long i) {
  return BF16 ? bf16_to_f32(__ldcg(static_cast<const unsigned short*>(p) + i)) : __ldcg(static_cast<const float*>(p) + i);
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, long long i, float v) {
  if (BF16)
    static_cast<uint16_t*>(p)[i] = f32_to_bf16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Where row `row` of the plan lives: false if it has no place (no sequence, a negative position, a page
// outside the cache). *owned: the row belongs to a sequence.
__device__ __forceinline__ bool kv4_place(const Kv4View& c, const Kv4Plan& p, int row, int& page, int& off, bool& owned,
                                          int* err) {
  const int b = kv4_seq_of(p, row);
  int r0, r1;
  kv4_rows(p, b, r0, r1, err);
  owned = row >= r0 && row < r1;
  if (!owned) return false;
  const int pos = kv4_len(p, c.page_log2, b, err) - (r1 - row);
  if (pos < 0) return false;
  page = __ldcg(p.table + (size_t)b * p.table_stride + (pos >> c.page_log2));
  off = pos & ((1 << c.page_log2) - 1);
  if (page < 0 || page >= c.pages) {
    set_error(err, COLI_E_RANGE);
    return false;
  }
  return true;
}

// Report row ranges and lengths that do not fit, whether or not a row of the call falls in them.
__device__ __forceinline__ void kv4_check_plan(const Kv4View& c, const Kv4Plan& p, long long item, int* err) {
  for (long long b = item; b < p.B; b += (long long)gridDim.x * kThreads) {
    int r0, r1;
    kv4_rows(p, (int)b, r0, r1, err);
    kv4_len(p, c.page_log2, (int)b, err);
  }
}

// Scale and offset of a group from this thread's four channels: the group is GL neighbouring lanes.
// Returns scale | offset << 16 and leaves the codes of the four channels in n.
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], int gl, uint32_t (&n)[4], int* err) {
  float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (!(fabsf(x[i]) < __int_as_float(0x7f800000))) {  // a value that is not finite makes the span so
      lo = -__int_as_float(0x7f800000);
      hi = __int_as_float(0x7f800000);
    }
  for (int m = 1; m < gl; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const float span = __fsub_rn(hi, lo);
  if (!(span < __int_as_float(0x7f800000))) {
    set_error(err, COLI_E_NONFINITE);
#pragma unroll
    for (int i = 0; i < 4; i++) n[i] = 8;
    return 0x7fc0u << 16;
  }
  uint32_t sb = f32_to_bf16_rn(__fmul_rn(span, 1.0f / 15.0f));
  if (sb < 0x0080u) sb = 0;  // below the smallest normal number
  const float s = bf16_to_f32((uint16_t)sb);
  const uint32_t ob = f32_to_bf16_rn(__fadd_rn(lo, __fmul_rn(8.0f, s)));
  const float o = bf16_to_f32((uint16_t)ob);
  const float inv = sb ? __frcp_rn(s) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float q = rintf(__fmul_rn(__fsub_rn(x[i], o), inv)) + 8.0f;
    n[i] = (uint32_t)fminf(fmaxf(q, 0.f), 15.f);
  }
  return sb | (ob << 16);
}

__device__ __forceinline__ uint32_t pack4(const uint32_t (&n)[4]) {
  return n[0] | (n[1] << 4) | (n[2] << 8) | (n[3] << 12);
}

// hd / 4 threads per (row, head): thread u holds the key channels 4 u .. 4 u + 3 and the value channels of
// the 16-bit piece (word u / 8, row u % 8); both lie in channels 32 (u / 8) .. + 31, so a group of gs
// channels is the same gs / 4 neighbouring lanes for keys and values.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(Kv4View c, Kv4Plan p, const void* k, long long k_stride,
                                                              const void* v, long long v_stride, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int tpr = c.hd / 4;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  kv4_check_plan(c, p, item, err);
  const int u = (int)(item % tpr);
  const long long rh = item / tpr;
  const bool in = rh < (long long)p.T * c.heads;
  const int row = in ? (int)(rh / c.heads) : 0, head = in ? (int)(rh % c.heads) : 0;
  int page = 0, off = 0;
  bool owned;
  const bool store = in && kv4_place(c, p, row, page, off, owned, err);
  const int i = u >> 3, r = u & 7;
  float xk[4] = {0.f, 0.f, 0.f, 0.f}, xv[4] = {0.f, 0.f, 0.f, 0.f};
  if (store) {
    const long long kb = row * k_stride + head * c.hd, vb = row * v_stride + head * c.hd;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      xk[j] = load1<BF16>(k, kb + 4 * u + j);
      xv[j] = load1<BF16>(v, vb + 32 * i + 16 * (j >> 1) + 2 * r + (j & 1));
    }
  }
  const int gl = tpr / c.ng;
  uint32_t nk[4], nv[4];
  const uint32_t pk = quantise(xk, gl, nk, err), pv = quantise(xv, gl, nv, err);
  if (!store) return;
  uint8_t* unit = const_cast<uint8_t*>(kv4_unit(c, page, head, off));
  const int t = off & 15, g = u / gl;
  *reinterpret_cast<uint16_t*>(unit + kv4_k_word(c.hd, t, i, r >> 1) + 2 * (r & 1)) = (uint16_t)pack4(nk);
  *reinterpret_cast<uint16_t*>(unit + kv4_v_at(c.hd, c.ng) + kv4_v_word(c.hd, t >> 1, r, i) + 2 * (t & 1)) =
      (uint16_t)pack4(nv);
  if (u % gl == 0) {
    *reinterpret_cast<uint32_t*>(unit + kv4_kscale_at(c.hd) + (t * c.ng + g) * 4) = pk;
    *reinterpret_cast<uint32_t*>(unit + kv4_vscale_at(c.hd, c.ng) + (t * c.ng + g) * 4) = pv;
  }
}

__device__ __forceinline__ float code_value(uint32_t par, uint32_t n) {
  const float s = __uint_as_float(par << 16), o = __uint_as_float(par & 0xffff0000u);
  return __fadd_rn(o, __fmul_rn(s, (float)((int)n - 8)));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(Kv4View c, Kv4Plan p, void* k, long long k_stride, void* v,
                                                            long long v_stride, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int tpr = c.hd / 4;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  kv4_check_plan(c, p, item, err);
  const int u = (int)(item % tpr);
  const long long rh = item / tpr;
  if (rh >= (long long)p.T * c.heads) return;
  const int row = (int)(rh / c.heads), head = (int)(rh % c.heads);
  int page = 0, off = 0;
  bool owned;
  const bool there = kv4_place(c, p, row, page, off, owned, err);
  if (!owned) return;
  const int i = u >> 3, r = u & 7, g = u / (tpr / c.ng);
  uint32_t nk = 0, nv = 0, pk = 0, pv = 0;
  if (there) {
    const uint8_t* unit = kv4_unit(c, page, head, off);
    const int t = off & 15;
    nk = __ldcg(reinterpret_cast<const unsigned short*>(unit + kv4_k_word(c.hd, t, i, r >> 1) + 2 * (r & 1)));
    nv = __ldcg(reinterpret_cast<const unsigned short*>(unit + kv4_v_at(c.hd, c.ng) + kv4_v_word(c.hd, t >> 1, r, i) +
                                                        2 * (t & 1)));
    pk = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_kscale_at(c.hd) + (t * c.ng + g) * 4));
    pv = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_vscale_at(c.hd, c.ng) + (t * c.ng + g) * 4));
  }
  const long long kb = row * k_stride + head * c.hd, vb = row * v_stride + head * c.hd;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    store1<BF16>(k, kb + 4 * u + j, code_value(pk, (nk >> (4 * j)) & 15u));
    store1<BF16>(v, vb + 32 * i + 16 * (j >> 1) + 2 * r + (j & 1), code_value(pv, (nv >> (4 * j)) & 15u));
  }
}

long long kv4_grid(const Kv4View& c, const Kv4Plan& p) {
  return ((long long)p.T * c.heads * (c.hd / 4) + kThreads - 1) / kThreads;
}

}  // namespace

int launch_kv4_append(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* k, long long k_stride, const void* v,
                      long long v_stride, int dtype) {
  const long long grid = kv4_grid(c, p);
  if (grid > 0x7fffffffll) return fail(ctx, COLI_E_INVAL, "kv4_append: too many rows for one call");
  ProfScope prof(ctx, COLI_KERNEL_CACHE);
  auto kern = dtype == COLI_DTYPE_BF16 ? kv4_append_kernel<true> : kv4_append_kernel<false>;
  cudaError_t e = launch_k(kern, (int)grid, kThreads, 0, ctx->stream, true, false, c, p, k, k_stride, v, v_stride,
                           ctx->d_status);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_append launch");
  return COLI_OK;
}

int launch_kv4_read(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, void* k, long long k_stride, void* v,
                    long long v_stride, int dtype) {
  const long long grid = kv4_grid(c, p);
  if (grid > 0x7fffffffll) return fail(ctx, COLI_E_INVAL, "kv4_read: too many rows for one call");
  ProfScope prof(ctx, COLI_KERNEL_CACHE);
  auto kern = dtype == COLI_DTYPE_BF16 ? kv4_read_kernel<true> : kv4_read_kernel<false>;
  cudaError_t e = launch_k(kern, (int)grid, kThreads, 0, ctx->stream, true, false, c, p, k, k_stride, v, v_stride,
                           ctx->d_status);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_read launch");
  return COLI_OK;
}

}  // namespace coli
