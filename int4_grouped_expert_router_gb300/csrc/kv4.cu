// Writing tokens into the 4-bit key/value cache and reading them back (layout: kv4.h).
//
// Both are bound by memory: the plain rows dominate. A warp takes 256 channels (eight neighbouring ones per lane) of up
// to four rows; of one row where there are too few to fill the device. All its loads are issued together, and the places
// of its rows are found by as many lanes at once. Codes are written as the layout gives them to a token: a whole word of
// keys, and of values the halves of two words. A token's halves lie eight sectors apart per head, so that a warp's rows
// are better neighbours in time than in channels (four rows of 256 channels 23.9 us, one row of 1024 27.9 us): two tokens
// of a pair store whole words, and the read finds the sectors of its other rows in the first-level cache. A group of gs
// channels is gs / 8 neighbouring lanes for keys and values alike. The two lanes whose channels share the value words of
// a token are two apart.
//
// Measured: 9198 ragged rows of 8 heads of 128 (bf16, gs 32) written and read back in 23.0 us (71 MB, 3.1 TB/s), a history
// of 36K rows of 4 heads of 64 read in 12.0 us (4.1 TB/s). Instructions and the chain plan, page, row bind them: the write
// fills 64 % of the issue slots and half of the ALU pipe, most of it the range, rounding and clamping of each channel, the
// read 58 %. CTAs of four warps took 3 % longer, of one or eight warps 10 %; eight rows a warp 10 to 20 %.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.h"
#include "pipe.h"

namespace coli {

namespace {

constexpr int kWarps = 2;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 256;  // channels of a warp's pass
// Passes of a warp whose loads are in flight together, where there are enough rows (registers: twice as many for bf16).
constexpr int most_slots(bool bf16) { return bf16 ? 4 : 2; }
constexpr float kInf = __builtin_huge_valf();

struct RowArgs {
  Kv4View c;
  Kv4Plan p;
  void* k;
  void* v;
  long long k_stride, v_stride;
  bool vec;    // rows start at a 16-byte boundary
  int groups;  // chunks (and warps) across a row
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

// Where a row lives.
struct Place {
  uint64_t at;  // offset in the cache of the unit of head 0
  int t;        // token of the unit
  bool owned;   // the row belongs to a sequence
  bool there;   // and has a place: a position that is not negative, a page of the cache
};

// The places of rows row0, row0 + 1, ..: lane l finds that of row0 + l, l < n (n at most kMostRows).
constexpr int kMostRows = 4;
__device__ __forceinline__ Place kv4_places(const RowArgs& a, int row0, int n) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  const bool mine = lane < n && row < a.p.T;
  Place at{0, 0, false, false};
  int b = row, r0 = row, r1 = row + 1, len = 0;
  if (!a.p.q_start) {
    if (mine) len = __ldcg(a.p.lens + b);
  } else if (a.p.B < 32) {
    // the whole plan in the warp's registers: one round trip
    const int start = lane <= a.p.B ? __ldcg(a.p.q_start + lane) : 0;
    const int length = lane < a.p.B ? __ldcg(a.p.lens + lane) : 0;
#pragma unroll
    for (int l = 0; l < kMostRows; l++) {
      const unsigned le = __ballot_sync(0xffffffffu, lane < a.p.B && start <= row0 + l);
      const int at_l = max(0, __popc(le) - 1);
      const int from = __shfl_sync(0xffffffffu, start, at_l), to = __shfl_sync(0xffffffffu, start, at_l + 1);
      const int have = __shfl_sync(0xffffffffu, length, at_l);
      if (lane == l) b = at_l, r0 = from, r1 = to, len = have;
    }
  } else {
    b = warp_seq_of(a.p, row0);
    if (mine) {
      while (b + 1 < a.p.B && __ldcg(a.p.q_start + b + 1) <= row) b++;  // a few steps: rows are neighbours
      r0 = __ldcg(a.p.q_start + b);
      r1 = __ldcg(a.p.q_start + b + 1);
      len = __ldcg(a.p.lens + b);
    }
  }
  // a range or a length that does not fit is reported by kv4_check_plan
  at.owned = mine && r0 >= 0 && r1 <= a.p.T && row >= r0 && row < r1;
  const long long most = kv4_most(a.p, a.c.page_log2);
  len = len < 0 ? 0 : len > most ? (int)most : len;
  const int pos = len - (r1 - row);
  if (!at.owned || pos < 0) return at;
  const int page = __ldcg(a.p.table + (size_t)b * a.p.table_stride + (pos >> a.c.page_log2));
  at.there = page >= 0 && page < a.c.pages;
  if (at.there) at.at = kv4_unit(a.c, page, 0, pos & ((1 << a.c.page_log2) - 1)) - a.c.base;
  at.t = pos & (kKvUnit - 1);
  if (!at.there) set_error(a.err, COLI_E_RANGE);
  return at;
}

// Lane l's place, in every lane.
__device__ __forceinline__ Place place_of(const Place& at, int l) {
  const int rest = __shfl_sync(0xffffffffu, (int)at.owned | (int)at.there << 1 | at.t << 2, l);
  return Place{__shfl_sync(0xffffffffu, at.at, l), rest >> 2, (rest & 1) != 0, (rest & 2) != 0};
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Two binary32 values as one 64-bit register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// A lane's eight channels as they lie in memory, and as binary32.
template <bool BF16>
struct Eight {
  uint32_t w[BF16 ? 4 : 8];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16)
      return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

template <bool BF16>
__device__ __forceinline__ Eight<BF16> load8(const void* p, long long at, bool vec) {
  Eight<BF16> x;
  constexpr int kWords = BF16 ? 4 : 8;
  if (vec) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = __ldcg(s + i / 4);
      x.w[i] = v.x, x.w[i + 1] = v.y, x.w[i + 2] = v.z, x.w[i + 3] = v.w;
    }
  } else if constexpr (BF16) {
    const unsigned short* s = static_cast<const unsigned short*>(p) + at;
#pragma unroll
    for (int i = 0; i < 4; i++) x.w[i] = __ldcg(s + 2 * i) | ((uint32_t)__ldcg(s + 2 * i + 1) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) x.w[i] = __ldcg(static_cast<const uint32_t*>(p) + at + i);
  }
  return x;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, long long at, bool vec, const Eight<BF16>& x) {
  if constexpr (BF16) {
    const auto& w = x.w;
    uint16_t* d = static_cast<uint16_t*>(p) + at;
    if (vec)
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    else
#pragma unroll
      for (int j = 0; j < 8; j++) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  } else {
    float* d = static_cast<float*>(p) + at;
    if (vec) {
      *reinterpret_cast<uint4*>(d) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
      *reinterpret_cast<uint4*>(d + 4) = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) d[j] = x[j];
    }
  }
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// The largest of a few channels and of their negatives; not a number if one of them is not. bf16 values are compared
// two at a time and travel as one register (largest, -least).
template <bool BF16>
struct Range {
  uint32_t m[BF16 ? 1 : 2];

  __device__ __forceinline__ void join(const Range& x) {
    if constexpr (BF16) {
      m[0] = bits(__hmax2_nan(as_bf162(m[0]), as_bf162(x.m[0])));
    } else {
#pragma unroll
      for (int i = 0; i < 2; i++) m[i] = __float_as_uint(max_nan(__uint_as_float(m[i]), __uint_as_float(x.m[i])));
    }
  }
  __device__ __forceinline__ Range across(int mask) const {  // that of lane ^ mask
    Range x;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); i++) x.m[i] = __shfl_xor_sync(0xffffffffu, m[i], mask);
    return x;
  }
  __device__ __forceinline__ float hi() const { return __uint_as_float(BF16 ? m[0] << 16 : m[0]); }
  __device__ __forceinline__ float lo() const { return -__uint_as_float(BF16 ? m[0] & 0xffff0000u : m[BF16 ? 0 : 1]); }
};

template <bool BF16>
__device__ __forceinline__ Range<BF16> range_of(const Eight<BF16>& x) {
  Range<BF16> r;
  if constexpr (BF16) {
    __nv_bfloat162 most = as_bf162(x.w[0]), least = most;
#pragma unroll
    for (int i = 1; i < 4; i++) {
      most = __hmax2_nan(most, as_bf162(x.w[i]));
      least = __hmin2_nan(least, as_bf162(x.w[i]));
    }
    // of the even channels, and of the odd ones
    const uint32_t neg = bits(least) ^ 0x80008000u;
    r.m[0] = __byte_perm(bits(most), neg, 0x5410);
    r.join({{__byte_perm(bits(most), neg, 0x7632)}});
  } else {
    float hi = x[0], lo = -x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) {
      hi = max_nan(hi, x[i]);
      lo = max_nan(lo, -x[i]);
    }
    r.m[0] = __float_as_uint(hi), r.m[1] = __float_as_uint(lo);
  }
  return r;
}

__device__ __forceinline__ uint32_t bf16_bits(float x) {  // of a number that is one
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// A group's scale | offset << 16, and 1 / scale, from its range.
template <bool BF16>
__device__ __forceinline__ uint32_t parameters(const Range<BF16>& x, float& inv, bool report, int* err) {
  const float lo = x.lo(), span = __fsub_rn(x.hi(), lo);
  uint32_t sb = 0, ob = 0x7fc0u;
  inv = 0.f;
  if (span < kInf) {
    sb = bf16_bits(__fmul_rn(span, 1.0f / 15.0f));
    if (sb < 0x0080u) sb = 0;  // below the smallest normal number
    const float s = __uint_as_float(sb << 16);
    ob = bf16_bits(__fadd_rn(lo, __fmul_rn(8.0f, s)));
    inv = sb ? __frcp_rn(s) : 0.f;
  } else if (report) {
    set_error(err, COLI_E_NONFINITE);
  }
  return sb | (ob << 16);
}

// Codes of eight channels, 4 bits each in order.
template <bool BF16>
__device__ __forceinline__ uint32_t codes(const Eight<BF16>& x, uint32_t par, float inv) {
  // a group that is not finite has no offset to take off
  const float o = (par & 0x7fff0000u) > 0x7f800000u ? 0.f : __uint_as_float(par & 0xffff0000u);
  // Adding 1.5 2^23 + 8 rounds the quotient to the nearest integer, ties to even, and leaves its bits as
  // 0x4b400000 + code, the code not yet clamped.
  if constexpr (BF16) {
    // A group that spans an ulp of its largest has codes within a few tens of 0..15 however o was rounded: they are
    // clamped two at a time in 16 bits, codes i and i + 4, as their places in the word are 16 bits apart. (The products
    // stay single: the compiler joins a product of pairs with the sum that follows, and its rounding would be lost.)
    const uint64_t neg_o = pack2(-o, -o), round = pack2(12582920.f, 12582920.f);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint64_t d = add2(pack2(x[2 * i], x[2 * i + 1]), neg_o);
      const float q0 = __fmul_rn(__uint_as_float((uint32_t)d), inv), q1 = __fmul_rn(__uint_as_float((uint32_t)(d >> 32)), inv);
      const uint64_t n = add2(pack2(q0, q1), round);
      c[2 * i] = (uint32_t)n, c[2 * i + 1] = (uint32_t)(n >> 32);
    }
    uint32_t n = 0;
#pragma unroll
    for (int i = 3; i >= 0; i--) n = n * 16u + __vimin_s16x2_relu(__byte_perm(c[i], c[i + 4], 0x5410), 0x000f000fu);
    return n;
  } else {
    // The quotient is clamped before it is rounded (the bounds are whole numbers); sixteenfold sums collect the codes,
    // and the constant's share comes off at the end.
    constexpr uint32_t kOnes = 0x11111111u;
    uint32_t n = 0;
#pragma unroll
    for (int i = 7; i >= 0; i--) {
      const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], o), inv), -8.f), 7.f);
      n = n * 16u + __float_as_uint(__fadd_rn(q, 12582920.f));
    }
    return n - 0x4b400000u * kOnes;
  }
}

// Keys and values of a row, in groups of GL neighbouring lanes: even lanes find the keys' scale and offset, odd lanes the
// values', and they exchange them. Returns the lane's own parameters.
template <bool BF16, int GL>
__device__ __forceinline__ uint32_t quantise(const Eight<BF16>& xk, const Eight<BF16>& xv, uint32_t& nk, uint32_t& nv, bool report,
                                             int* err) {
  static_assert(GL >= 2, "a group has lanes of both kinds");
  const bool odd = threadIdx.x & 1;
  const Range<BF16> k = range_of(xk), v = range_of(xv);
  Range<BF16> mine = odd ? v : k;
  mine.join((odd ? k : v).across(1));
#pragma unroll
  for (int s = 2; s < GL; s <<= 1) mine.join(mine.across(s));
  float inv;
  const uint32_t par = parameters(mine, inv, report, err);
  const uint32_t par2 = __shfl_xor_sync(0xffffffffu, par, 1);
  const float inv2 = __shfl_xor_sync(0xffffffffu, inv, 1);
  nk = codes(xk, odd ? par2 : par, odd ? inv2 : inv);
  nv = codes(xv, odd ? par : par2, odd ? inv : inv2);
  return par;
}

// A lane's place in its chunk: head and the lane's number u within it.
template <int HD>
struct Spot {
  int head, u;
  bool in;
  __device__ __forceinline__ Spot(int chunk, int heads) {
    const int x = chunk * kChunk + (threadIdx.x & 31) * 8;
    head = x / HD;
    u = x % HD / 8;
    in = head < heads;
  }
};

// A warp's slots: one chunk of kSlots rows.
template <int kSlots>
struct Share {
  int row0, chunk;
  __device__ __forceinline__ Share(const RowArgs& a) {
    const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    row0 = item / a.groups * kSlots;
    chunk = item % a.groups;
  }
};

template <bool BF16, int HD, int NG, int kSlots>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(RowArgs a) {
  constexpr int kGl = HD / NG / 8;  // lanes of a group
  griddep_launch_dependents();
  griddep_wait();
  kv4_check_plan(a);
  const Share<kSlots> w(a);
  if (w.row0 >= a.p.T) return;  // uniform in the warp
  const Spot<HD> s(w.chunk, a.c.heads);
  Eight<BF16> xk[kSlots] = {}, xv[kSlots] = {};
#pragma unroll
  for (int n = 0; n < kSlots; n++) {
    const long long row = w.row0 + n;
    if (row < a.p.T && s.in) {
      xk[n] = load8<BF16>(a.k, row * a.k_stride + s.head * HD + 8 * s.u, a.vec);
      xv[n] = load8<BF16>(a.v, row * a.v_stride + s.head * HD + 8 * s.u, a.vec);
    }
  }
  const Place places = kv4_places(a, w.row0, kSlots);
  const uint32_t head_at = s.head * ((uint32_t)(1 << (a.c.page_log2 - 4)) * kv4_unit_bytes(HD, NG));
  const int i = s.u >> 2, c = s.u & 3, upper = c >> 1, r = 4 * (c & 1) + 2 * upper;
  Place to[kSlots];
  uint32_t two[kSlots];
#pragma unroll
  for (int n = 0; n < kSlots; n++) {
    to[n] = place_of(places, n);
    if (!to[n].there) continue;  // uniform
    uint32_t nk, nv;
    const uint32_t par = quantise<BF16, kGl>(xk[n], xv[n], nk, nv, s.in, a.err);
    // A token's half of a value word holds two channels below 16 of a run of 32 and the two 16 above: bytes of two
    // lanes, each of which puts two of the four words together.
    const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? nv & 0xffffu : nv >> 16, 2);
    two[n] = upper ? __byte_perm(nv, other, 0x3524) : __byte_perm(nv, other, 0x5140);
    if (!s.in) continue;
    const int t = to[n].t;
    uint8_t* unit = a.c.base + to[n].at + head_at;
    *reinterpret_cast<uint32_t*>(unit + kv4_k_word(HD, t, i, c)) = nk;
    if (s.u % kGl < 2)
      *reinterpret_cast<uint32_t*>(unit + (s.u & 1 ? kv4_vscale_at(HD, NG) : kv4_kscale_at(HD)) + (t * NG + s.u / kGl) * 4) = par;
  }
  if (!s.in) return;
  // the value words: whole where the other token is the next row
  bool done = false;
#pragma unroll
  for (int n = 0; n < kSlots; n++) {
    if (done || !to[n].there) {
      done = false;
      continue;
    }
    const int t = to[n].t;
    uint8_t* v = a.c.base + to[n].at + head_at + kv4_v_at(HD, NG);
    uint8_t *v0 = v + kv4_v_word(HD, t >> 1, r, i), *v1 = v + kv4_v_word(HD, t >> 1, r + 1, i);
    if (n + 1 < kSlots && (t & 1) == 0 && to[n + 1].there && to[n + 1].at == to[n].at && to[n + 1].t == t + 1) {
      *reinterpret_cast<uint32_t*>(v0) = __byte_perm(two[n], two[n + 1], 0x5410);
      *reinterpret_cast<uint32_t*>(v1) = __byte_perm(two[n], two[n + 1], 0x7632);
      done = true;
    } else {
      reinterpret_cast<uint16_t*>(v0)[t & 1] = (uint16_t)two[n];
      reinterpret_cast<uint16_t*>(v1)[t & 1] = (uint16_t)(two[n] >> 16);
    }
  }
}

// o + s (n - 8) of a word's eight codes, rounded once: the product is exact in binary32, and bf16 takes one multiply-add
// of its own type, for two channels.
template <bool BF16>
__device__ __forceinline__ Eight<BF16> values(uint32_t w, uint32_t par) {
  Eight<BF16> x;
  if constexpr (BF16) {
    const __nv_bfloat162 s = as_bf162(__byte_perm(par, 0, 0x1010)), o = as_bf162(__byte_perm(par, 0, 0x3232));
    const __nv_bfloat162 bias = __floats2bfloat162_rn(-136.f, -136.f);
    uint32_t v[4];
#pragma unroll
    for (int m = 0; m < 4; m++) {  // channels m and m + 4
      const uint32_t t = ((w >> (4 * m)) & 0x000f000fu) | 0x43004300u;  // 128 + n in bf16
      v[m] = bits(__hfma2(__hadd2(as_bf162(t), bias), s, o));
    }
#pragma unroll
    for (int i = 0; i < 4; i++) x.w[i] = __byte_perm(v[2 * i & 3], v[(2 * i & 3) + 1], i < 2 ? 0x5410 : 0x7632);
  } else {
    const float s = __uint_as_float(par << 16), o = __uint_as_float(par & 0xffff0000u);
    const __half2 bias = __floats2half2_rn(1032.f, 1032.f);
#pragma unroll
    for (int m = 0; m < 4; m++) {
      const uint32_t t = ((w >> (4 * m)) & 0x000f000fu) | 0x64006400u;  // 1024 + n in 16 bits
      const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&t), bias);
      x.w[m] = __float_as_uint(fmaf(s, __low2float(n), o));
      x.w[m + 4] = __float_as_uint(fmaf(s, __high2float(n), o));
    }
  }
  return x;
}

template <bool BF16, int HD, int NG, int kSlots>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(RowArgs a) {
  constexpr int kGl = HD / NG / 8;
  griddep_launch_dependents();
  griddep_wait();
  kv4_check_plan(a);
  const Share<kSlots> w(a);
  if (w.row0 >= a.p.T) return;
  const Spot<HD> s(w.chunk, a.c.heads);
  const Place places = kv4_places(a, w.row0, kSlots);
  const uint32_t head_at = s.head * ((uint32_t)(1 << (a.c.page_log2 - 4)) * kv4_unit_bytes(HD, NG));
  const int i = s.u >> 2, c = s.u & 3, r = 4 * (c & 1) + (c & 2), g = s.u / kGl;
  uint32_t nk[kSlots], nv[kSlots], pk[kSlots], pv[kSlots];
  bool owned[kSlots];
  // through the first-level cache: the rows of a warp, and of its neighbours, are tokens that share sectors
#pragma unroll
  for (int n = 0; n < kSlots; n++) {
    const Place from = place_of(places, n);
    owned[n] = from.owned;
    nk[n] = nv[n] = pk[n] = pv[n] = 0;
    if (!s.in || !from.there) continue;
    const int t = from.t;
    const uint8_t* unit = a.c.base + from.at + head_at;
    const uint8_t* v = unit + kv4_v_at(HD, NG) + 2 * (t & 1);
    nk[n] = *reinterpret_cast<const uint32_t*>(unit + kv4_k_word(HD, t, i, c));
    nv[n] = *reinterpret_cast<const unsigned short*>(v + kv4_v_word(HD, t >> 1, r, i)) |
            ((uint32_t)*reinterpret_cast<const unsigned short*>(v + kv4_v_word(HD, t >> 1, r + 1, i)) << 16);
    pk[n] = *reinterpret_cast<const uint32_t*>(unit + kv4_kscale_at(HD) + (t * NG + g) * 4);
    pv[n] = *reinterpret_cast<const uint32_t*>(unit + kv4_vscale_at(HD, NG) + (t * NG + g) * 4);
  }
  const bool upper = s.u & 2;  // as in the append
#pragma unroll
  for (int n = 0; n < kSlots; n++) {
    const long long row = w.row0 + n;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, __byte_perm(nv[n], 0, upper ? 0x4420 : 0x4431), 2);
    const uint32_t mine = __byte_perm(nv[n], other, upper ? 0x3154 : 0x5420);
    if (!s.in || !owned[n]) continue;
    store8<BF16>(a.k, row * a.k_stride + s.head * HD + 8 * s.u, a.vec, values<BF16>(nk[n], pk[n]));
    store8<BF16>(a.v, row * a.v_stride + s.head * HD + 8 * s.u, a.vec, values<BF16>(mine, pv[n]));
  }
}

template <bool READ, bool BF16, int SLOTS>
void (*kernel_of(int hd, int ng))(RowArgs) {
#define COLI_KV4_KERNEL(HD, NG) (READ ? kv4_read_kernel<BF16, HD, NG, SLOTS> : kv4_append_kernel<BF16, HD, NG, SLOTS>)
  if (hd == 64) return ng == 1 ? COLI_KV4_KERNEL(64, 1) : COLI_KV4_KERNEL(64, 2);
  if (hd == 128) return ng == 1 ? COLI_KV4_KERNEL(128, 1) : ng == 2 ? COLI_KV4_KERNEL(128, 2) : COLI_KV4_KERNEL(128, 4);
  return ng == 2 ? COLI_KV4_KERNEL(256, 2) : COLI_KV4_KERNEL(256, 4);
#undef COLI_KV4_KERNEL
}

template <bool READ>
int launch_rows(coli_ctx* ctx, const char* who, const Kv4View& c, const Kv4Plan& p, void* k, long long k_stride, void* v,
                long long v_stride, int dtype) {
  RowArgs a{c, p, k, v, k_stride, v_stride};
  const int per16 = dtype == COLI_DTYPE_BF16 ? 8 : 4;
  a.vec = (((uintptr_t)k | (uintptr_t)v) & 15) == 0 && k_stride % per16 == 0 && v_stride % per16 == 0;
  // several slots a warp where that still gives every SM's schedulers a few warps
  const bool bf16 = dtype == COLI_DTYPE_BF16;
  const int chunks = (c.heads * c.hd + kChunk - 1) / kChunk;
  const int slots = (long long)p.T * chunks >= (long long)most_slots(bf16) * 8 * ctx->num_sms ? most_slots(bf16) : 1;
  a.groups = chunks;
  a.err = ctx->d_status;
  const long long grid = (((long long)p.T + slots - 1) / slots * chunks + kWarps - 1) / kWarps;
  if (grid * kWarps > 0x7fffffffll) return fail(ctx, COLI_E_INVAL, std::string(who) + ": too many rows for one call");
  ProfScope prof(ctx, COLI_KERNEL_CACHE);
  auto kern = bf16 ? (slots > 1 ? kernel_of<READ, true, most_slots(true)>(c.hd, c.ng) : kernel_of<READ, true, 1>(c.hd, c.ng))
                   : (slots > 1 ? kernel_of<READ, false, most_slots(false)>(c.hd, c.ng) : kernel_of<READ, false, 1>(c.hd, c.ng));
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
