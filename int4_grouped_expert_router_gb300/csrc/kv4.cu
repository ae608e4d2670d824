// Writing tokens into the 4-bit key/value cache and reading them back (layout: kv4.h).
//
// Both are bound by memory: the plain rows dominate. A warp takes one row's next 512 channels (up to four
// chunks of 128, four neighbouring channels per lane, all loads issued first), finds the row's place once,
// and writes or reads the codes as the 16-bit pieces that the layout gives a token. In a chunk, lane group
// u / 8 holds the 32 channels of one code word index, so a group of gs channels is gs / 4 neighbouring
// lanes for keys and values alike, and the two halves of a value piece are four lanes apart.
#include <cuda_bf16.h>

#include "kv4.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 128;  // channels of a warp's pass
constexpr int kChunks = 4;   // passes whose loads are in flight together
constexpr float kInf = __builtin_huge_valf();

struct RowArgs {
  Kv4View c;
  Kv4Plan p;
  void* k;
  void* v;
  long long k_stride, v_stride;
  bool vec;    // rows start at a boundary of four elements
  int groups;  // warps per row
  int* err;
};

// Report row ranges and lengths that do not fit, whether or not a row of the call falls in them.
__device__ __forceinline__ void kv4_check_plan(const RowArgs& a) {
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.p.B; b += gridDim.x * kThreads) {
    int r0, r1;
    kv4_rows(a.p, b, r0, r1, a.err);
    kv4_len(a.p, a.c.page_log2, b, a.err);
  }
}

// The last sequence b with q_start[b] <= row, found by a whole warp, 32 entries at a time. Whatever
// q_start holds, the result is a sequence; kv4_place checks that it owns the row.
__device__ __forceinline__ int warp_seq_of(const Kv4Plan& p, int row) {
  if (!p.q_start) return row;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldcg(p.q_start + at) <= row);
    lo += max(0, __popc(le) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Where row `row` of the plan lives: false if it has no place (no sequence, a negative position, a page
// outside the cache). owned: the row belongs to a sequence.
__device__ __forceinline__ bool kv4_place(const RowArgs& a, int row, int& page, int& off, bool& owned) {
  const int b = warp_seq_of(a.p, row);
  int r0, r1;
  kv4_rows(a.p, b, r0, r1, a.err);
  owned = row >= r0 && row < r1;
  if (!owned) return false;
  const int pos = kv4_len(a.p, a.c.page_log2, b, a.err) - (r1 - row);
  if (pos < 0) return false;
  page = __ldcg(a.p.table + (size_t)b * a.p.table_stride + (pos >> a.c.page_log2));
  off = pos & ((1 << a.c.page_log2) - 1);
  if (page < 0 || page >= a.c.pages) {
    set_error(a.err, COLI_E_RANGE);
    return false;
  }
  return true;
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Least and largest of a group's channels (GL neighbouring lanes, four channels each); not a number if one
// of them is not. bf16 values travel as one register, the largest and the negated least.
template <bool BF16, int GL>
__device__ __forceinline__ void group_range(const float (&x)[4], float& lo, float& hi) {
  hi = max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
  lo = max_nan(max_nan(-x[0], -x[1]), max_nan(-x[2], -x[3]));
  if constexpr (BF16) {
    __nv_bfloat162 m = __floats2bfloat162_rn(lo, hi);  // exact
#pragma unroll
    for (int s = 1; s < GL; s <<= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&m), s);
      m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&o));
    }
    lo = -__low2float(m);
    hi = __high2float(m);
  } else {
#pragma unroll
    for (int s = 1; s < GL; s <<= 1) {
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
      lo = max_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
    }
    lo = -lo;
  }
}

// Codes of this lane's four channels, 4 bits each in order; the group's scale | offset << 16.
template <bool BF16, int GL>
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], uint32_t& par, bool report, int* err) {
  float lo, hi;
  group_range<BF16, GL>(x, lo, hi);
  const float span = __fsub_rn(hi, lo);
  uint32_t sb = 0, ob = 0x7fc0u;
  float inv = 0.f, o = 0.f;
  if (span < kInf) {
    sb = f32_to_bf16_rn(__fmul_rn(span, 1.0f / 15.0f));
    if (sb < 0x0080u) sb = 0;  // below the smallest normal number
    const float s = bf16_to_f32((uint16_t)sb);
    ob = f32_to_bf16_rn(__fadd_rn(lo, __fmul_rn(8.0f, s)));
    o = bf16_to_f32((uint16_t)ob);
    inv = sb ? __frcp_rn(s) : 0.f;
  } else if (report) {
    set_error(err, COLI_E_NONFINITE);
  }
  par = sb | (ob << 16);
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    // clamped before it is rounded (the bounds are whole numbers); adding 1.5 2^23 + 8 rounds to the nearest
    // integer, ties to even, and leaves it, 8 added, in the low bits
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], o), inv), -8.f), 7.f);
    const uint32_t code = inv == 0.f ? 8u : __float_as_uint(__fadd_rn(q, 12582920.f)) & 15u;
    n |= code << (4 * i);
  }
  return n;
}

template <bool BF16>
__device__ __forceinline__ void load4(const void* p, long long i, bool vec, float (&x)[4]) {
  if constexpr (BF16) {
    const unsigned short* s = static_cast<const unsigned short*>(p) + i;
    if (vec) {
      const uint2 w = __ldcg(reinterpret_cast<const uint2*>(s));
      x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) x[j] = bf16_to_f32(__ldcg(s + j));
    }
  } else {
    const float* s = static_cast<const float*>(p) + i;
    if (vec) {
      const float4 w = __ldcg(reinterpret_cast<const float4*>(s));
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) x[j] = __ldcg(s + j);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store4(void* p, long long i, bool vec, const float (&x)[4]) {
  if constexpr (BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    const uint32_t w[2] = {*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)};
    uint16_t* d = static_cast<uint16_t*>(p) + i;
    if (vec)
      *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    else
#pragma unroll
      for (int j = 0; j < 4; j++) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  } else {
    float* d = static_cast<float*>(p) + i;
    if (vec)
      *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    else
#pragma unroll
      for (int j = 0; j < 4; j++) d[j] = x[j];
  }
}

// A lane's place in its chunk: head and the lane's number u within it.
template <int HD>
struct Spot {
  int head, u;
  bool in;
  __device__ __forceinline__ Spot(int chunk, int heads) {
    const int x = chunk * kChunk + (threadIdx.x & 31) * 4;
    head = x / HD;
    u = x % HD / 4;
    in = head < heads;
  }
};

template <bool BF16, int HD, int NG>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(RowArgs a) {
  constexpr int kGl = HD / NG / 4;  // lanes of a group
  griddep_launch_dependents();
  griddep_wait();
  kv4_check_plan(a);
  const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int row = item / a.groups, chunk0 = item % a.groups * kChunks;
  if (row >= a.p.T) return;  // uniform in the warp
  float xk[kChunks][4], xv[kChunks][4];
#pragma unroll
  for (int n = 0; n < kChunks; n++) {
    const Spot<HD> s(chunk0 + n, a.c.heads);
    if (s.in) {
      load4<BF16>(a.k, row * a.k_stride + s.head * HD + 4 * s.u, a.vec, xk[n]);
      load4<BF16>(a.v, row * a.v_stride + s.head * HD + 4 * s.u, a.vec, xv[n]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) xk[n][j] = xv[n][j] = 0.f;
    }
  }
  int page = 0, off = 0;
  bool owned;
  if (!kv4_place(a, row, page, off, owned)) return;  // uniform in the warp
  uint8_t* at = const_cast<uint8_t*>(kv4_unit(a.c, page, 0, off));
  const uint32_t head_bytes = (uint32_t)(1 << (a.c.page_log2 - 4)) * kv4_unit_bytes(HD, NG);
  const int t = off & 15;
#pragma unroll
  for (int n = 0; n < kChunks; n++) {
    if ((chunk0 + n) * kChunk >= a.c.heads * HD) break;  // uniform
    const Spot<HD> s(chunk0 + n, a.c.heads);
    uint32_t pk, pv;
    const uint32_t nk = quantise<BF16, kGl>(xk[n], pk, s.in, a.err), nv = quantise<BF16, kGl>(xv[n], pv, s.in, a.err);
    // value pieces: the low byte from the lane with channels 0..15 of the 32, the high byte from 16..31;
    // each of the two lanes puts one of its two rows together
    const int i = s.u >> 3, half = s.u >> 2 & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, half ? nv & 0xffu : nv >> 8, 4);
    const uint32_t piece = half ? other | (nv & 0xff00u) : (nv & 0xffu) | (other << 8);
    if (!s.in) continue;
    uint8_t* unit = at + s.head * head_bytes;
    *reinterpret_cast<uint16_t*>(unit + kv4_k_word(HD, t, i, s.u >> 1 & 3) + 2 * (s.u & 1)) = (uint16_t)nk;
    *reinterpret_cast<uint16_t*>(unit + kv4_v_at(HD, NG) + kv4_v_word(HD, t >> 1, 2 * (s.u & 3) + half, i) + 2 * (t & 1)) =
        (uint16_t)piece;
    if (s.u % kGl == 0) {
      const int g = s.u / kGl;
      *reinterpret_cast<uint32_t*>(unit + kv4_kscale_at(HD) + (t * NG + g) * 4) = pk;
      *reinterpret_cast<uint32_t*>(unit + kv4_vscale_at(HD, NG) + (t * NG + g) * 4) = pv;
    }
  }
}

// o + s (n - 8): the product is exact, so one rounding.
__device__ __forceinline__ void values(uint32_t n, uint32_t par, float (&x)[4]) {
  const float s = __uint_as_float(par << 16), o = __uint_as_float(par & 0xffff0000u);
#pragma unroll
  for (int j = 0; j < 4; j++)
    x[j] = fmaf(s, __uint_as_float(0x4b000000u | (n >> (4 * j) & 15u)) - 8388616.f, o);
}

template <bool BF16, int HD, int NG>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(RowArgs a) {
  constexpr int kGl = HD / NG / 4;
  griddep_launch_dependents();
  griddep_wait();
  kv4_check_plan(a);
  const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int row = item / a.groups, chunk0 = item % a.groups * kChunks;
  if (row >= a.p.T) return;
  int page = 0, off = 0;
  bool owned;
  const bool there = kv4_place(a, row, page, off, owned);
  if (!owned) return;
  const uint8_t* at = kv4_unit(a.c, page, 0, off);
  const uint32_t head_bytes = (uint32_t)(1 << (a.c.page_log2 - 4)) * kv4_unit_bytes(HD, NG);
  const int t = off & 15;
  uint32_t nk[kChunks], nv[kChunks], pk[kChunks], pv[kChunks];
#pragma unroll
  for (int n = 0; n < kChunks; n++) {
    const Spot<HD> s(chunk0 + n, a.c.heads);
    nk[n] = nv[n] = pk[n] = pv[n] = 0;
    if (!s.in || !there) continue;
    const int i = s.u >> 3, half = s.u >> 2 & 1, g = s.u / kGl;
    const uint8_t* unit = at + s.head * head_bytes;
    nk[n] = __ldcg(reinterpret_cast<const unsigned short*>(unit + kv4_k_word(HD, t, i, s.u >> 1 & 3) + 2 * (s.u & 1)));
    nv[n] = __ldcg(reinterpret_cast<const unsigned short*>(
        unit + kv4_v_at(HD, NG) + kv4_v_word(HD, t >> 1, 2 * (s.u & 3) + half, i) + 2 * (t & 1)));
    pk[n] = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_kscale_at(HD) + (t * NG + g) * 4));
    pv[n] = __ldcg(reinterpret_cast<const uint32_t*>(unit + kv4_vscale_at(HD, NG) + (t * NG + g) * 4));
  }
#pragma unroll
  for (int n = 0; n < kChunks; n++) {
    if ((chunk0 + n) * kChunk >= a.c.heads * HD) break;  // uniform
    const Spot<HD> s(chunk0 + n, a.c.heads);
    const int half = s.u >> 2 & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, half ? nv[n] & 0xffu : nv[n] >> 8, 4);
    const uint32_t mine = half ? other | (nv[n] & 0xff00u) : (nv[n] & 0xffu) | (other << 8);
    if (!s.in) continue;
    float x[4];
    values(nk[n], pk[n], x);
    store4<BF16>(a.k, row * a.k_stride + s.head * HD + 4 * s.u, a.vec, x);
    values(mine, pv[n], x);
    store4<BF16>(a.v, row * a.v_stride + s.head * HD + 4 * s.u, a.vec, x);
  }
}

template <bool READ, bool BF16>
void (*kernel_of(int hd, int ng))(RowArgs) {
#define COLI_KV4_KERNEL(HD, NG) (READ ? kv4_read_kernel<BF16, HD, NG> : kv4_append_kernel<BF16, HD, NG>)
  if (hd == 64) return ng == 1 ? COLI_KV4_KERNEL(64, 1) : COLI_KV4_KERNEL(64, 2);
  if (hd == 128) return ng == 1 ? COLI_KV4_KERNEL(128, 1) : ng == 2 ? COLI_KV4_KERNEL(128, 2) : COLI_KV4_KERNEL(128, 4);
  return ng == 2 ? COLI_KV4_KERNEL(256, 2) : COLI_KV4_KERNEL(256, 4);
#undef COLI_KV4_KERNEL
}

template <bool READ>
int launch_rows(coli_ctx* ctx, const char* who, const Kv4View& c, const Kv4Plan& p, void* k, long long k_stride, void* v,
                long long v_stride, int dtype) {
  const uintptr_t four = dtype == COLI_DTYPE_BF16 ? 8 : 16;
  RowArgs a{c, p, k, v, k_stride, v_stride};
  a.vec = (((uintptr_t)k | (uintptr_t)v) % four) == 0 && k_stride % 4 == 0 && v_stride % 4 == 0;
  a.groups = (c.heads * c.hd + kChunk * kChunks - 1) / (kChunk * kChunks);
  a.err = ctx->d_status;
  const long long grid = ((long long)p.T * a.groups + kWarps - 1) / kWarps;
  if (grid * kWarps > 0x7fffffffll) return fail(ctx, COLI_E_INVAL, std::string(who) + ": too many rows for one call");
  ProfScope prof(ctx, COLI_KERNEL_CACHE);
  auto kern = dtype == COLI_DTYPE_BF16 ? kernel_of<READ, true>(c.hd, c.ng) : kernel_of<READ, false>(c.hd, c.ng);
  cudaError_t e = launch_k(kern, (int)grid, kThreads, 0, ctx->stream, true, false, a);
  if (e != cudaSuccess) return cuda_fail(ctx, e, who);
  return COLI_OK;
}

}  // namespace

int launch_kv4_append(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, const void* k, long long k_stride, const void* v,
                      long long v_stride, int dtype) {
  return launch_rows<false>(ctx, "kv4_append", c, p, const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride, dtype);
}

int launch_kv4_read(coli_ctx* ctx, const Kv4View& c, const Kv4Plan& p, void* k, long long k_stride, void* v,
                    long long v_stride, int dtype) {
  return launch_rows<true>(ctx, "kv4_read", c, p, k, k_stride, v, v_stride, dtype);
}

}  // namespace coli
