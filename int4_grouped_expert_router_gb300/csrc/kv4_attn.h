// Attention over the 4-bit key/value cache (layout: kv4.h), for decode steps and the few rows of drafts.
//
// For a query row q at position p of its sequence and the visible positions t,
//   x_t = scale sum_g [ s_tg q_g . (n_tg - 8) + o_tg sum(q_g) ],   out = sum_t a_t V_t / sum_t a_t,
//   a_t = exp(x_t - max x),   sum_t a_t V_t = sum_t (a_t s_tg) (n_tg - 8) + sum_t a_t o_tg,
// one pass over the tokens with a running maximum and sum. The codes enter the matrix instructions as the small
// integers that they are (exact in 16 bits): a group's scale and offset are applied to the score of its token, and to
// the weight a_t before V. Queries enter in 16 bits after a power of two has brought a row's largest to 2^14 (bf16
// ones then are exact down to 2^-27 of it: half of them also take a factor 1/16); f32 queries and weights enter as a sum
// of two 16-bit values.
//
// What bounds it: the cache's bytes, read once (a key/value head's codes serve all of its query heads), and beside
// them the instructions that unpack codes and weigh tokens, about 340 per 16 tokens of a head (hd = 128, one group):
// with every copy left out the kernel takes as long, with the arithmetic left out 0.6 of its time.
//
// Work split. An item is (sequence, key/value head, tile of 8 NT query rows); its tokens are cut into stages of 64,
// and all items' stages, end to end, are dealt out evenly and contiguously to a grid that fills the device, each item
// counting kItemCost stages more: whatever the lengths, every CTA has the same work. An item that spans CTAs leaves
// partial (maximum, sum, output) triples in the context's memory, and whoever arrives last adds them up in CTA order, so that
// results do not depend on who is last.
//
// In a CTA a producer warp fills a ring of stages with bulk copies, a run of units of a page each (64 tokens are
// 8.7 KB at hd = 128, gs = 128: codes and scales of keys and values together), and four consumer warps take one unit
// (16 tokens) of each stage, with their own running maximum and sum; they are joined in shared memory when the item
// ends. Three CTAs share an SM: one joins while the others compute (one CTA of twelve warps took 1.4 times as long on
// a batch of 64).
// Four CTAs without producers, each warp fetching its own units, took 1.05 to 1.13 times as long; 32 query rows a
// tile instead of two tiles of 16 (30 rows over up to 20011 tokens) 124 us instead of 112.
//
// Consumer, per unit: S^T = K q^T with m16n8k16 (rows = 16 tokens, columns = 8 query rows: group sizes up to 8 fill
// the instruction, where queries as rows would leave half of it empty), the softmax on the accumulators, the weights
// transposed in registers (movmatrix), O^T += V^T a (rows = 16 channels).
//
// Measured (bf16, hd 128, a copy's rate being 6782 GB/s): 64 requests of up to 8192 tokens, 8 heads of 8, gs 64:
// 84 us, 3.6 TB/s; 131071 tokens of one request, gs 128: 44 us, 3.3 TB/s; a request of 1003 tokens: 10 us, of which
// the launch, the dealing out, the queries and the joining of 16 parts are all but one.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "kv4.h"
#include "pipe.h"

namespace coli {

struct AttnArgs {
  Kv4View c;
  Kv4Plan p;
  const void* q;
  long long q_stride;
  int group;      // query heads per key/value head
  float scale;
  int window;
  void* out;
  long long out_stride;
  bool vec;       // q rows start at 16-byte boundaries
  bool vec_out;   // out rows start at a boundary of four values
  float* part;    // partial results: 2 per CTA, each kRows x HD outputs and kRows (maximum, sum) pairs
  int* count;     // arrivals: 2 per CTA for the run of parts whose sum its slot takes, then 1 per CTA for the runs of an item
  int* err;
  uint64_t wait_ns;
  bool withhold;  // test hook: the call's first copy is withheld, and the waits on it give up
};

// One translation unit per type of the activations (kv4_attn.cu, kv4_attn_f32.cu): they compile side by side.
int launch_attn_bf16(coli_ctx* ctx, AttnArgs& a);
int launch_attn_f32(coli_ctx* ctx, AttnArgs& a);

namespace {

constexpr int kStageUnits = 4;                    // consumer warps, and units of a stage
constexpr int kStageTok = kStageUnits * kKvUnit;  // tokens of a stage
constexpr int kConsumers = kStageUnits * 32;
constexpr int kAttnThreads = kConsumers + 32;
// A row's running maximum follows the scores only when one exceeds it by this much (log2), so weights stay below
// 2^kSlack: moving it costs a pass over the unit's sums, and at kSlack = 1 did so often enough to take a fifth of
// the time. The scales (or values) that a weight meets in 16 bits are kept below 2^9.
constexpr float kSlack = 6.f;
constexpr float kTopScale = 512.f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kGroup = 8;  // parts summed at once
// What an item costs beside its stages (queries in, the warps' results joined), in stages: it counts in the shares,
// ahead of the item's first stage.
#ifndef COLI_KV4_ITEM_COST
#define COLI_KV4_ITEM_COST 4
#endif
constexpr int kItemCost = COLI_KV4_ITEM_COST;

template <int HD, int NG, int NT, bool F32>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kWords = HD / 32;       // code words of a token a lane holds (keys); as many per token pair (values)
  static constexpr int kWpg = kWords / NG;     // of which a group takes
  static constexpr int kIw = kWords < 4 ? kWords : 4;
  static constexpr int kMt = HD / 16;          // 16-channel tiles of the output
  static constexpr int kPad = HD + 4;          // floats of a row in the join buffer: no bank conflicts at 8-byte stores
  static constexpr uint32_t kUnit = kv4_unit_bytes(HD, NG);
  static constexpr uint32_t kStage = kStageUnits * kUnit;
  // Values enter the product dequantised where several tiles of rows share the work of it (bf16: 11 bits); otherwise as
  // codes, with a group's scale on the weight.
  static constexpr bool kDeq = !F32 && NT > 1;
  // Key codes enter as they lie (0..15) for bf16 queries; centred for f32 ones, whose scores would lose two bits to the
  // larger sums.
  static constexpr bool kRawK = !F32;
  static constexpr float kOdd = kRawK ? 0.0625f : 1.f;           // queries of codes at bit 4, which count sixteenfold
  static constexpr float kUnitK = kRawK ? 16777216.f : 1.f;      // a code is this many times what enters
  // Value codes enter as they are (0..15). The instruction cuts its accumulator off instead of rounding it, and codes
  // that are not centred make the sum large beside the result, so that what is cut shows there, always downward: hence
  // codes at bit 4, and sums that leave the accumulator after kSumUnits. Balanced values then cancel to 2^-22 of eight
  // steps (2^-18.5 with codes as they lie and 64 units, where 131071 tokens came out 0.07 % too low; that took 80 us for
  // the batch of 64, this 84, centred codes 86).
  static constexpr bool kRawV = !F32 && NT == 1;
  static constexpr float kTop = kDeq ? 16384.f : kTopScale;  // dequantised values and weights are rounded apart
  static constexpr int kSumUnits = 16;  // units after which a sum moves to shared memory
  static constexpr int kCtas = HD == 256 ? (NT == 1 ? 2 : 1) : NT == 1 ? 3 : 2;  // resident per SM (registers)
  static constexpr uint32_t kJoin = kStageUnits * kRows * (kPad + 2) * 4;
  static constexpr uint32_t kQ = NT * (HD / 16) * 32 * 8 * (F32 ? 2 : 1);
  static constexpr uint32_t kBudget = (kCtas == 3 ? 74 : kCtas == 2 ? 112 : 200) * 1024;
  static constexpr int kRoom = (int)((kBudget - kJoin - kQ - 1024) / kStage);
  static constexpr int kStages = kRoom > 12 ? 12 : kRoom;
  static constexpr uint32_t kSmem = kStages * kStage + kJoin + kQ;
  static_assert(kStages >= 3, "the ring needs a few stages");
};

// Where an item starts in the dealt-out stages, and what a CTA needs to know of it.
struct Item {
  int b, head, tile;     // sequence, key/value head, tile of query rows
  int r0, m, len;        // the sequence's first row, its rows and its length
  int first, stages;     // first stage of 64 tokens, number of stages (at least 1)
};

__device__ __forceinline__ void load_seq(const Kv4View& c, const Kv4Plan& p, int window, Item& it, int* err) {
  int r1;
  kv4_rows(p, it.b, it.r0, r1, err);
  it.m = r1 - it.r0;
  it.len = kv4_len(p, c.page_log2, it.b, err);
  // the first row's window starts the sequence's visible part
  it.first = kv4_from(it.len - it.m, window) / kStageTok;
  it.stages = max(1, (it.len + kStageTok - 1) / kStageTok - it.first);
}

__device__ __forceinline__ int tiles_of(int m, int group, int rows) { return (int)(((long long)m * group + rows - 1) / rows); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes of word w as two registers' worth each: pair m of (w >> 4 m) & 0x000f000f, as the 16-bit
// integers n - 8. The bits 0x6400 put a nibble at the end of 1024's mantissa (one logic operation), and at
// bit 4 as sixteen times itself, which the multiply-add undoes.
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&a)[4]) {
  const __half2 bias = __floats2half2_rn(1032.f, 1032.f);
  const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f), bias16 = __floats2half2_rn(-72.f, -72.f);
  const uint32_t w8 = w >> 8;
  uint32_t t[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u, (w8 & 0x000f000fu) | 0x64006400u,
                   (w8 & 0x00f000f0u) | 0x64006400u};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __half2 h = *reinterpret_cast<__half2*>(&t[i]);
    const __half2 v = (i & 1) ? __hfma2(h, sixteenth, bias16) : __hsub2(h, bias);
    a[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// The same pairs as they lie, one logic operation each: a nibble at the end of a 16-bit float's mantissa is the
// subnormal number n 2^-24, at bit 4 n 2^-20, which the matrix instruction takes as they are. Its sum, however, is cut off
// some 24 bits below the operands' smallest normal number times the other factor, whatever leading zeros a subnormal one
// has: at the mantissa's end 18 to 19 bits of the sum are left.
__device__ __forceinline__ void expand_raw(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t w8 = w >> 8;
  a[0] = w & 0x000f000fu;
  a[1] = w & 0x00f000f0u;
  a[2] = w8 & 0x000f000fu;
  a[3] = w8 & 0x00f000f0u;
}

// The same pairs as n 2^-20, all at bit 4: so the sum keeps 22 bits.
__device__ __forceinline__ void expand_raw4(uint32_t w, uint32_t (&a)[4]) {
  a[0] = (w << 4) & 0x00f000f0u;
  a[1] = w & 0x00f000f0u;
  a[2] = (w >> 4) & 0x00f000f0u;
  a[3] = (w >> 8) & 0x00f000f0u;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from a zero accumulator.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// N words of a lane from shared memory (32-bit addresses: no 64-bit arithmetic in the loop).
__device__ __forceinline__ void lds4(uint32_t p, uint32_t* w) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p) : "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    lds4(p, w);
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p) : "memory");
  } else {
    static_assert(N == 1, "1, 2 or 4 words");
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p) : "memory");
  }
}

// A lane's code words of one 16-token key row or value pair row, kv4.h: iw words per access, accesses
// `apart` bytes from each other.
template <int WORDS>
__device__ __forceinline__ void lds_codes(uint32_t p, int apart, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS <= 4) {
    lds_words(p, w);
  } else {
    lds4(p, w);
    lds4(p + apart, w + 4);
  }
}

template <bool F32>
__device__ __forceinline__ void load_q8(const void* q, size_t at, float (&v)[8], bool vec) {
  if constexpr (F32) {
    const float* s = static_cast<const float*>(q) + at;
    if (vec) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(s)), b = __ldcg(reinterpret_cast<const float4*>(s) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = __ldcg(s + i);
    }
  } else {
    const unsigned short* s = static_cast<const unsigned short*>(q) + at;
    if (vec) {
      const uint4 a = __ldcg(reinterpret_cast<const uint4*>(s));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; i++) v[2 * i] = lo_bf16(w[i]), v[2 * i + 1] = hi_bf16(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = bf16_to_f32(__ldcg(s + i));
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store4(void* out, size_t at, float4 v, bool vec) {
  if constexpr (F32) {
    float* o = static_cast<float*>(out) + at;
    if (vec)
      *reinterpret_cast<float4*>(o) = v;
    else
      o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    const uint16_t h[4] = {f32_to_bf16_rn(v.x), f32_to_bf16_rn(v.y), f32_to_bf16_rn(v.z), f32_to_bf16_rn(v.w)};
    if (vec)
      *reinterpret_cast<uint2*>(o) = make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
    else
      o[0] = h[0], o[1] = h[1], o[2] = h[2], o[3] = h[3];
  }
}

template <int HD, int NG, int NT, bool F32>
__global__ void __launch_bounds__(kAttnThreads, Cfg<HD, NG, NT, F32>::kCtas) kv4_attn_kernel(AttnArgs a) {
  using C = Cfg<HD, NG, NT, F32>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* s_join = reinterpret_cast<float*>(smem + C::kStages * C::kStage);  // [4][kRows][kPad], then maxima and sums
  float* s_m = s_join + kStageUnits * C::kRows * C::kPad;                   // [4][kRows]
  float* s_l = s_m + kStageUnits * C::kRows;
  uint2* s_q = reinterpret_cast<uint2*>(smem + C::kStages * C::kStage + C::kJoin);  // query fragments [hi, lo][NT][HD / 16][32]
  __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages];
  __shared__ long long s_sum[kAttnThreads / 32];
  __shared__ long long s_at;
  __shared__ int s_last;
  __shared__ Item s_item;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; i++) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kStageUnits);
    }
    mbar_fence_init();
  }
  griddep_launch_dependents();
  griddep_wait();

  // ---- deal the stages out: total, then the sequence in which this CTA's share starts ----
  const int heads = a.c.heads;
  Item t;
  auto stages_in = [&](int b) -> long long {
    t.b = b;
    load_seq(a.c, a.p, a.window, t, a.err);
    return (long long)tiles_of(t.m, a.group, C::kRows) * heads * (t.stages + kItemCost);
  };
  long long total = 0, own = 0;
  for (int b = tid; b < a.p.B; b += kAttnThreads) total += own = stages_in(b);
  const bool once = a.p.B <= kAttnThreads;  // then a thread still has its sequence
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kAttnThreads / 32; i++) total += s_sum[i];
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long w0 = per * blockIdx.x, w1 = w0 + per < total ? w0 + per : total;
  if (w0 >= w1) return;  // uniform in the CTA; nothing in flight
  long long before = 0;
  for (int base = 0; base < a.p.B; base += kAttnThreads) {
    const int b = base + tid;
    const long long mine = once ? own : b < a.p.B ? stages_in(b) : 0;
    long long inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long off = before, all = 0;
    for (int i = 0; i < kAttnThreads / 32; i++) {
      if (i < warp) off += s_sum[i];
      all += s_sum[i];
    }
    const long long start = off + inc - mine;
    if (mine > 0 && start <= w0 && w0 < start + mine) {
      s_item = t;
      s_at = start;
    }
    before += all;
    if (before > w0) break;  // uniform
  }
  __syncthreads();

  // ---- the cursor that producer and consumers walk on their own ----
  Item it = s_item;
  const long long local = w0 - s_at;  // stages of this sequence before the share
  const int tiles0 = tiles_of(it.m, a.group, C::kRows);
  const long long item0 = local / (it.stages + kItemCost);
  it.head = (int)(item0 / tiles0);
  it.tile = (int)(item0 % tiles0);
  // within the item; below 0: in its cost. w counts stages and costs: stage s of the item at `item_at` is at
  // item_at + kItemCost + s.
  int stage = (int)(local % (it.stages + kItemCost)) - kItemCost;
  long long w = w0;
  auto next_item = [&]() {  // after the last stage of an item; w < w1 guarantees that there is one
    if (++it.tile < tiles_of(it.m, a.group, C::kRows)) return;
    it.tile = 0;
    if (++it.head < heads) return;
    it.head = 0;
    do {
      it.b++;
      load_seq(a.c, a.p, a.window, it, a.err);
    } while (it.m == 0 && it.b + 1 < a.p.B);
  };

  if (warp == kStageUnits) {
    // ------------------------------------ producer ------------------------------------
    // A lane per stage, several stages at a time: their page numbers are one round trip, and each lane issues as
    // soon as its slot is free.
    const uint64_t policy = l2_evict_first_policy();
    const int page_tok = 1 << a.c.page_log2;
    const int per_copy = min(kStageUnits, page_tok / kKvUnit);  // units
    const size_t page_bytes = (size_t)heads * (page_tok / kKvUnit) * C::kUnit;
    int slot = 0;
    uint32_t phase = 1;
    bool lost = false;
    int fills = 0;  // of this lane's slot (lane < kStages)
    while (!lost) {
      if (stage < 0) w -= stage, stage = 0;
      if (w >= w1) break;
      const int n = (int)min((long long)min(C::kStages, it.stages - stage), w1 - w);
      const int tok = (it.first + stage + lane) * kStageTok;
      const int units = lane < n ? min(kStageUnits, max(0, (it.len - tok + kKvUnit - 1) / kKvUnit)) : 0;
      const uint8_t* src[kStageUnits];
#pragma unroll
      for (int k = 0; k < kStageUnits; k++) {
        if (k * per_copy >= units) continue;
        const int at = tok + k * per_copy * kKvUnit;
        int pg = __ldcg(a.p.table + (size_t)it.b * a.p.table_stride + (at >> a.c.page_log2));
        if (pg < 0 || pg >= a.c.pages) {
          if (at + per_copy * kKvUnit > kv4_from(it.len - it.m, a.window)) set_error(a.err, COLI_E_RANGE);
          pg = 0;  // some page of the cache in its place; no row sees a page that its window has left
        }
        src[k] = a.c.base + pg * page_bytes + (uint32_t)(it.head * (page_tok / kKvUnit) + (at & (page_tok - 1)) / kKvUnit) * C::kUnit;
      }
      int mine = slot + lane;
      uint32_t my_phase = phase;
      if (mine >= C::kStages) {
        mine -= C::kStages;
        my_phase ^= 1;
      }
      const bool held = a.withhold && w == kItemCost && lane == 0;
      bool done = lane >= n || held;
      const uint64_t t0 = globaltimer_ns();
      while (!done) {
        if (mbar_test_wait(&s_empty[mine], my_phase)) {
          mbar_arrive_expect_tx(&s_full[mine], units * C::kUnit);
#pragma unroll
          for (int k = 0; k < kStageUnits; k++)
            if (k * per_copy < units)
              bulk_g2s_stream(ring + mine * C::kStage + k * per_copy * C::kUnit, src[k],
                              min(per_copy, units - k * per_copy) * C::kUnit, &s_full[mine], policy);
          done = true;
        } else if (globaltimer_ns() - t0 > a.wait_ns) {
          set_error(a.err, COLI_E_TIMEOUT);
          lost = done = true;  // what was issued is still awaited by the consumers
        }
      }
      // the slots of this round that were filled, from `slot` on: this lane's is `lane - slot` from there
      const unsigned filled = __ballot_sync(0xffffffffu, lane < n && !lost && !held);
      if (lane < C::kStages && (filled >> ((lane - slot + C::kStages) % C::kStages) & 1)) fills++;
      lost = __any_sync(0xffffffffu, lost);
      slot += n;
      if (slot >= C::kStages) {
        slot -= C::kStages;
        phase ^= 1;
      }
      w += n;
      stage += n;
      if (stage == it.stages) {
        stage = -kItemCost;
        if (w < w1) next_item();
      }
    }
    // no copy is in flight when the CTA ends, even if the consumers gave one up
    if (lane < C::kStages && fills > 0) mbar_wait(&s_full[lane], (fills - 1) & 1);
    return;
  }

  // -------------------------------------- consumers --------------------------------------
  const int r = lane >> 2, cc = lane & 3;
  const uint32_t ring_at = smem_u32(ring);
  int slot = 0;
  uint32_t phase = 0;
  bool alive = true;
  while (true) {
    // ---- a segment: this CTA's stages of one item ----
    if (stage < 0) w -= stage, stage = 0;
    if (w >= w1) break;
    const long long item_at = w - stage;  // where the item's first stage is in what was dealt out
    const int n_here = (int)min((long long)(it.stages - stage), w1 - w);
    const int tile_row = it.tile * C::kRows;
    const int rows_all = it.m * a.group;  // this sequence's query rows per key/value head
    const int row_n = min(C::kRows, rows_all - tile_row);

    // queries: fragments of 16-bit integers-friendly values (each row scaled by a power of two so that its
    // largest element lies in [2^14, 2^15): bf16 elements down to 2^-27 of it stay exact, kOdd counted), their sums per
    // group, and the factor that takes a row's scores to log2 units.
    float fac[NT][2], sumq[NT][2][NG];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int row = tile_row + nt * 8 + r;
      float v[C::kWords][8];
      float amax = 0.f;
      bool fin = true;
      if (nt * 8 + r < row_n) {
        const size_t at = (size_t)((it.r0 + row / a.group) * a.q_stride) + (size_t)(it.head * a.group + row % a.group) * HD;
#pragma unroll
        for (int i = 0; i < C::kWords; i++) {
          load_q8<F32>(a.q, at + 32 * i + 8 * cc, v[i], a.vec);
#pragma unroll
          for (int j = 0; j < 8; j++) {
            amax = fmaxf(amax, fabsf(v[i][j]));
            fin = fin && fabsf(v[i][j]) < kInf;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kWords; i++)
#pragma unroll
          for (int j = 0; j < 8; j++) v[i][j] = 0.f;
      }
      if (!fin) {
        set_error(a.err, COLI_E_NONFINITE);
        amax = kInf;
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^(14 - floor(log2 amax)), its exponent kept within what binary32 has
      const int ex = min(253, max(1, 127 + 14 + 127 - (int)(__float_as_uint(amax) >> 23)));
      float mult = amax == 0.f ? 1.f : __uint_as_float((uint32_t)ex << 23);
      const float inv = amax == 0.f ? 1.f : __uint_as_float((uint32_t)(254 - ex) << 23);
      if (a.scale < 0.f) mult = -mult;
      if (!(amax < kInf)) mult = __uint_as_float(0x7fc00000u);
      float sum[NG];
#pragma unroll
      for (int g = 0; g < NG; g++) sum[g] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kWords; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
          v[i][j] *= mult;
          sum[i / C::kWpg] += v[i][j];
        }
#pragma unroll
      for (int g = 0; g < NG; g++) {
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
#pragma unroll
        for (int e = 0; e < 2; e++) sumq[nt][e][g] = (1.f / C::kUnitK) * __shfl_sync(0xffffffffu, sum[g], (2 * cc + e) * 4);
      }
      // not 0: minus infinity stays it
      const float f = fmaxf(fabsf(a.scale) * 1.4426950408889634f * inv * C::kUnitK, 1e-37f);
#pragma unroll
      for (int e = 0; e < 2; e++) {
        fac[nt][e] = __shfl_sync(0xffffffffu, f, (2 * cc + e) * 4);
        const int qr = min(tile_row + nt * 8 + 2 * cc + e, rows_all - 1);  // rows past the end count like the last
        pos[nt][e] = it.len - it.m + qr / a.group;
      }
      // step 2 i + h of the contraction: k slots (2 c, 2 c + 1) and (2 c + 8, 2 c + 9) are channels
      // (2 h, 2 h + 4) and (2 h + 1, 2 h + 5) of this lane's eight. Warp w keeps the steps of its share.
#pragma unroll
      for (int i = 0; i < C::kWords; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          if ((2 * i + h) % kStageUnits != warp) continue;
          const int at = (nt * (HD / 16) + 2 * i + h) * 32 + lane;
          const float v1 = v[i][2 * h + 1] * C::kOdd, v5 = v[i][2 * h + 5] * C::kOdd;
          const uint32_t b0 = pack_half2(v[i][2 * h], v[i][2 * h + 4]), b1 = pack_half2(v1, v5);
          s_q[at] = make_uint2(b0, b1);
          if constexpr (F32) {
            const __half2 h0 = *reinterpret_cast<const __half2*>(&b0), h1 = *reinterpret_cast<const __half2*>(&b1);
            s_q[NT * (HD / 16) * 32 + at] =
                make_uint2(pack_half2(v[i][2 * h] - __low2float(h0), v[i][2 * h + 4] - __high2float(h0)),
                           pack_half2(v1 - __low2float(h1), v5 - __high2float(h1)));
          }
        }
    }
    named_sync(1, kConsumers);
    float o[NT][C::kMt][4], lsum[NT][2], bias[NT][2][NG], mf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int i = 0; i < C::kMt; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) o[nt][i][j] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; e++) {
        lsum[nt][e] = 0.f;
        mf[nt][e] = -kInf;
#pragma unroll
        for (int g = 0; g < NG; g++) bias[nt][e][g] = 0.f;
      }
    }
    // value scales (dequantised: values) are multiplied by vmul, a power of two that keeps them below kTop; it only
    // shrinks, and the outputs with it.
    float vmul = __uint_as_float(253u << 23), eight = 8.f / vmul;
    bool stashed = false;                                  // part of the sums lies in the join buffer
    uint32_t nan_groups = 0;                               // dequantised: by row and group, a value seen is not finite
    float* stash = s_join + warp * C::kRows * C::kPad + 2 * r;
    const int pos_min = it.len - it.m + tile_row / a.group;  // first row's position
    const int pos_max = it.len - it.m + (tile_row + row_n - 1) / a.group;
    const int lo_max = kv4_from(pos_max, a.window), lo_min = kv4_from(pos_min, a.window);

    // One unit; `masked`: some row does not see some token of it.
    auto process = [&](auto masked, uint32_t unit, int t0) {
      constexpr bool kMasked = decltype(masked)::value;
      const uint32_t codes = unit + lane * (C::kIw * 4);
      uint32_t kp[2][NG], vp[2][NG];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        lds_words(unit + kv4_kscale_at(HD) + (r + 8 * h) * NG * 4, kp[h]);
        lds_words(unit + kv4_vscale_at(HD, NG) + (r + 8 * h) * NG * 4, vp[h]);
        if (kMasked && (t0 + r + 8 * h >= it.len || t0 + r + 8 * h < lo_min)) {  // tokens that no row sees hold anything
#pragma unroll
          for (int g = 0; g < NG; g++) vp[h][g] = 0;
        }
      }
      // ---- scores ----
      float x[NT][4];
      {
        uint32_t kw[2][C::kWords];
        lds_codes(codes, 1024, kw[0]);
        lds_codes(codes + 128 * C::kIw, 1024, kw[1]);
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int j = 0; j < 4; j++) x[nt][j] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; g++) {
          float acc[2][NT][4];  // two chains: even and odd steps
#pragma unroll
          for (int i = g * C::kWpg; i < (g + 1) * C::kWpg; i++) {
            uint32_t a0[4], a1[4];
            if constexpr (C::kRawK) {
              expand_raw(kw[0][i], a0);
              expand_raw(kw[1][i], a1);
            } else {
              expand(kw[0][i], a0);
              expand(kw[1][i], a1);
            }
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
              for (int nt = 0; nt < NT; nt++) {
                const uint2 b = s_q[(nt * (HD / 16) + 2 * i + h) * 32 + lane];
                if (i == g * C::kWpg)
                  mma16816_zero(acc[h][nt], a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1], b.x, b.y);
                else
                  mma16816(acc[h][nt], a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1], b.x, b.y);
                if constexpr (F32) {
                  const uint2 l = s_q[((NT + nt) * (HD / 16) + 2 * i + h) * 32 + lane];
                  mma16816(acc[h][nt], a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1], l.x, l.y);
                }
              }
          }
          const float ks[2] = {lo_bf16(kp[0][g]), lo_bf16(kp[1][g])};
          float ko[2] = {hi_bf16(kp[0][g]), hi_bf16(kp[1][g])};
          if constexpr (C::kRawK) {  // of code 0
            ko[0] = fmaf(-8.f, ks[0], ko[0]);
            ko[1] = fmaf(-8.f, ks[1], ko[1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 4; j++)
              x[nt][j] = fmaf(ks[j >> 1], acc[0][nt][j] + acc[1][nt][j], fmaf(ko[j >> 1], sumq[nt][j & 1][g], x[nt][j]));
        }
      }
      if constexpr (kMasked) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            // (the difference may wrap for a negative position, which sees nothing anyhow)
            const int t = t0 + r + 8 * (j >> 1), p = pos[nt][j & 1];
            if (t > p || (a.window > 0 && t <= (int)((uint32_t)p - (uint32_t)a.window))) x[nt][j] = -kInf;
          }
      }
      // ---- running maximum: moves only when a score passes it by kSlack ----
      float y[NT][4], most = -kInf;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
#pragma unroll
        for (int j = 0; j < 4; j++) y[nt][j] = fmaf(fac[nt][j & 1], x[nt][j], -mf[nt][j & 1]);
        most = max3(max3(most, y[nt][0], y[nt][1]), y[nt][2], y[nt][3]);
      }
      // largest value scale (dequantised: bound of the values, not a number or infinite if one is not finite) of the unit
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int g = 0; g < NG; g++)
          top = C::kDeq ? max_nan(top, fmaf(8.f, lo_bf16(vp[h][g]), fabsf(hi_bf16(vp[h][g])))) : fmaxf(top, lo_bf16(vp[h][g]));
      if (__any_sync(0xffffffffu, most > kSlack || !(top * vmul < C::kTop))) {
        if (C::kDeq && !(top < kInf)) {
          // what is not finite stays out of the factor and the product, and is noted in the rows that see it
          top = 0.f;
#pragma unroll
          for (int h = 0; h < 2; h++) {
            uint32_t bad = 0;
#pragma unroll
            for (int g = 0; g < NG; g++) {
              if (kv4_broken(vp[h][g]))
                bad |= 1u << g;
              else
                top = fmaxf(top, fmaf(8.f, lo_bf16(vp[h][g]), fabsf(hi_bf16(vp[h][g]))));
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (!kMasked || x[nt][2 * h + e] != -kInf) nan_groups |= bad << ((nt * 2 + e) * NG);
          }
        }
        const float seen = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        float shrink = 1.f;
        if (seen * vmul >= C::kTop) {
          // the power of two that brings seen into the upper half of [0, kTop)
          const int ex = min(253, max(1, (int)(__float_as_uint(C::kTop) >> 23) - 1 + 127 - (int)(__float_as_uint(seen) >> 23)));
          const float now = __uint_as_float((uint32_t)ex << 23);
          shrink = now / vmul;
          vmul = now;
          eight = 8.f / vmul;
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float mx = fmaxf(x[nt][e], x[nt][2 + e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float now = mx == -kInf ? mf[nt][e] : fmaxf(mf[nt][e], fac[nt][e] * mx);
            const float f = mf[nt][e] == -kInf ? 1.f : exp2_fast(mf[nt][e] - now);
            mf[nt][e] = now;
            lsum[nt][e] *= f;
#pragma unroll
            for (int g = 0; g < NG; g++) bias[nt][e][g] *= f;
#pragma unroll
            for (int i = 0; i < C::kMt; i++) {
              o[nt][i][e] *= f * shrink;
              o[nt][i][2 + e] *= f * shrink;
            }
            if (C::kRawV && stashed) {
#pragma unroll 1
              for (int i = 0; i < C::kMt; i++) {
                float2* at = reinterpret_cast<float2*>(stash + (nt * 8 + 2 * cc + e) * C::kPad + 16 * i);
                *at = make_float2(at->x * (f * shrink), at->y * (f * shrink));
              }
            }
#pragma unroll
            for (int j = e; j < 4; j += 2) y[nt][j] = fmaf(fac[nt][e], x[nt][j], -now);
          }
      }
      // ---- weights, transposed into B fragments ----
      float pr[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          pr[nt][j] = exp2_fast(y[nt][j]);
          if (kMasked && x[nt][j] == -kInf) pr[nt][j] = 0.f;  // a row that has seen nothing has no maximum
        }
        lsum[nt][0] += pr[nt][0] + pr[nt][2];
        lsum[nt][1] += pr[nt][1] + pr[nt][3];
      }
      constexpr int kPg = C::kDeq ? 1 : NG;  // weights per group
      uint32_t pb[NT][kPg][2];
      [[maybe_unused]] uint32_t pl[F32 ? NT : 1][kPg][2];
      if constexpr (C::kDeq) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int h = 0; h < 2; h++) pb[nt][0][h] = transpose8x8(pack_half2(pr[nt][2 * h] * kTopScale, pr[nt][2 * h + 1] * kTopScale));
      } else {
        // A bf16 call's weight enters the product as h = round(a s vmul) in 11 bits. The offset takes the same
        // rounded weight, as h (o / (s vmul)): rounding it then scales the token's V as a whole, however far o is
        // from it. The quotient gets a correction step, so that it is exact where V = 0 is. Where the scale is
        // nothing beside the largest, the offset is V. With the 22 bits of an f32 call's weights a itself serves.
#pragma unroll
        for (int g = 0; g < NG; g++) {
          float vs[2], vo[2];
          bool faint[2];
#pragma unroll
          for (int h = 0; h < 2; h++) {
            vs[h] = lo_bf16(vp[h][g]) * vmul;
            vo[h] = hi_bf16(vp[h][g]);
            faint[h] = F32 || vs[h] < 9.3132257e-10f;  // 2^-30
            if (!F32) {
              const float inv = rcp_fast(vs[h]), q = vo[h] * inv;
              const float quotient = fmaf(fmaf(-q, vs[h], vo[h]), inv, q) - eight;  // of code 0
              vo[h] = faint[h] ? vo[h] : quotient;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const float pv[2] = {pr[nt][2 * h] * vs[h], pr[nt][2 * h + 1] * vs[h]};
              const uint32_t hi = pack_half2(pv[0], pv[1]);
              const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
              const float kept[2] = {__low2float(hh), __high2float(hh)};
              pb[nt][g][h] = transpose8x8(hi);
              if constexpr (F32) pl[nt][g][h] = transpose8x8(pack_half2(pv[0] - kept[0], pv[1] - kept[1]));
#pragma unroll
              for (int e = 0; e < 2; e++) {
                float off = vo[h];
                if (kMasked && x[nt][2 * h + e] == -kInf) off = 0.f;  // an unseen NaN stays unseen
                bias[nt][e][g] = fmaf(faint[h] ? pr[nt][2 * h + e] : kept[e], off, bias[nt][e][g]);
              }
            }
        }
      }
      // ---- output ----
      {
        const uint32_t vb = codes + kv4_v_at(HD, NG);
        uint32_t vw[2][C::kWords];
        lds_codes(vb, 512, vw[0]);
        lds_codes(vb + 4 * HD, 512, vw[1]);
        [[maybe_unused]] __half2 s[C::kDeq ? 2 : 1][NG], off[C::kDeq ? 2 : 1][NG];
        if constexpr (C::kDeq) {
#pragma unroll
          for (int h = 0; h < 2; h++) {  // tokens 2 c, 2 c + 1 and the eight after
            uint32_t p0[NG], p1[NG];
            const uint32_t at = unit + kv4_vscale_at(HD, NG) + (2 * cc + 8 * h) * NG * 4;
            lds_words(at, p0);
            lds_words(at + NG * 4, p1);
            const int t = t0 + 2 * cc + 8 * h;
            const bool live0 = !kMasked || (t < it.len && t >= lo_min), live1 = !kMasked || (t + 1 < it.len && t + 1 >= lo_min);
#pragma unroll
            for (int g = 0; g < NG; g++) {
              const float o0 = hi_bf16(p0[g]), o1 = hi_bf16(p1[g]);
              s[h][g] = __floats2half2_rn(live0 ? lo_bf16(p0[g]) * vmul : 0.f, live1 ? lo_bf16(p1[g]) * vmul : 0.f);
              off[h][g] = __floats2half2_rn(live0 && fabsf(o0) < kInf ? o0 * vmul : 0.f, live1 && fabsf(o1) < kInf ? o1 * vmul : 0.f);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < C::kWords; i++) {
          const int g = i / C::kWpg;
          uint32_t a0[4], a1[4];
          if constexpr (C::kRawV) {
            expand_raw4(vw[0][i], a0);
            expand_raw4(vw[1][i], a1);
          } else {
            expand(vw[0][i], a0);
            expand(vw[1][i], a1);
          }
          if constexpr (C::kDeq) {
#pragma unroll
            for (int m = 0; m < 4; m++) {
              const __half2 v0 = __hfma2(*reinterpret_cast<const __half2*>(&a0[m]), s[0][g], off[0][g]);
              const __half2 v1 = __hfma2(*reinterpret_cast<const __half2*>(&a1[m]), s[1][g], off[1][g]);
              a0[m] = *reinterpret_cast<const uint32_t*>(&v0);
              a1[m] = *reinterpret_cast<const uint32_t*>(&v1);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              float(&d)[4] = o[nt][2 * i + h];
              const int pg = C::kDeq ? 0 : g;
              if constexpr (F32) {
                // the instruction's own accumulator is cut, not rounded: a unit's sum is formed from zero and
                // added in binary32
                float t[4];
                mma16816_zero(t, a0[2 * h], a0[2 * h + 1], a1[2 * h], a1[2 * h + 1], pl[nt][pg][0], pl[nt][pg][1]);
                mma16816(t, a0[2 * h], a0[2 * h + 1], a1[2 * h], a1[2 * h + 1], pb[nt][pg][0], pb[nt][pg][1]);
#pragma unroll
                for (int j = 0; j < 4; j++) d[j] += t[j];
              } else {
                mma16816(d, a0[2 * h], a0[2 * h + 1], a1[2 * h], a1[2 * h + 1], pb[nt][pg][0], pb[nt][pg][1]);
              }
            }
        }
      }
    };

    for (int n = 0; n < n_here; n++, w++, stage++) {
      const int t0 = (it.first + stage) * kStageTok + warp * kKvUnit;
      if (alive && !mbar_wait_suspend(&s_full[slot], phase, a.wait_ns)) {
        set_error(a.err, COLI_E_TIMEOUT);
        alive = false;  // whatever the ring holds is used: the result is void, but nothing hangs
      }
      const uint32_t unit = ring_at + slot * C::kStage + warp * C::kUnit;
      if (t0 <= pos_max && t0 + kKvUnit > lo_min) {  // some row of the tile sees some token of the unit
        if (t0 + kKvUnit - 1 > pos_min || t0 < lo_max)
          process(std::true_type{}, unit, t0);
        else
          process(std::false_type{}, unit, t0);
      }
      if (C::kRawV && n % C::kSumUnits == C::kSumUnits - 1) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int e = 0; e < 2; e++)
#pragma unroll
            for (int i = 0; i < C::kMt; i++) {
              float2* at = reinterpret_cast<float2*>(stash + (nt * 8 + 2 * cc + e) * C::kPad + 16 * i);
              const float2 had = stashed ? *at : make_float2(0.f, 0.f);
              *at = make_float2(had.x + o[nt][i][e], had.y + o[nt][i][2 + e]);
              o[nt][i][e] = o[nt][i][2 + e] = 0.f;
            }
        stashed = true;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[slot]);
      if (++slot == C::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }

    // ---- join the four warps ----
    // exact: powers of two, one after the other for values as codes (their product may not be a number)
    constexpr float kUnscale = C::kRawV ? 1048576.f : 1.f;
    const float vinv = (C::kDeq ? 1.f / kTopScale : 1.f) / vmul;
    if constexpr (C::kDeq)
      for (int s = 4; s < 32; s <<= 1) nan_groups |= __shfl_xor_sync(0xffffffffu, nan_groups, s);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float l = lsum[nt][e];
        for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
#pragma unroll
        for (int g = 0; g < NG; g++) {
          float t = bias[nt][e][g];
          for (int s = 4; s < 32; s <<= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
          bias[nt][e][g] = t;
        }
        const int row = nt * 8 + 2 * cc + e;
        if (r == 0) {
          s_m[warp * C::kRows + row] = mf[nt][e];
          s_l[warp * C::kRows + row] = l;
        }
        float* dst = s_join + (warp * C::kRows + row) * C::kPad + 2 * r;
#pragma unroll
        for (int i = 0; i < C::kMt; i++) {
          const int g = (i / 2) / C::kWpg;
          const float add = !C::kDeq ? bias[nt][e][g] : nan_groups >> ((nt * 2 + e) * NG + g) & 1 ? __uint_as_float(0x7fc00000u) : 0.f;
          float2* at = reinterpret_cast<float2*>(dst + 16 * i);
          const float2 had = C::kRawV && stashed ? *at : make_float2(0.f, 0.f);
          *at = make_float2(fmaf((had.x + o[nt][i][e]) * kUnscale, vinv, add), fmaf((had.y + o[nt][i][2 + e]) * kUnscale, vinv, add));
        }
      }
    named_sync(1, kConsumers);
    const bool whole = n_here == it.stages;
    const bool starts_here = item_at >= w0;
    float* part = a.part + (size_t)(2 * blockIdx.x + starts_here) * C::kRows * (HD + 2);
    auto out_at = [&](int row) {
      const int q = tile_row + row;
      return (size_t)((it.r0 + q / a.group) * a.out_stride) + (size_t)(it.head * a.group + q % a.group) * HD;
    };
    for (int i = tid; i < row_n * (HD / 4); i += kConsumers) {
      const int row = i / (HD / 4), d = (i % (HD / 4)) * 4;
      float mm = -kInf;
#pragma unroll
      for (int k = 0; k < kStageUnits; k++) mm = fmaxf(mm, s_m[k * C::kRows + row]);
      float l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kStageUnits; k++) {
        const float f = s_m[k * C::kRows + row] == -kInf ? 0.f : exp2_fast(s_m[k * C::kRows + row] - mm);
        // a warp without a maximum saw nothing, or only what is not a number
        const float lk = s_l[k * C::kRows + row];
        const float4 v = *reinterpret_cast<const float4*>(s_join + (k * C::kRows + row) * C::kPad + d);
        if (f != 0.f || lk != 0.f) {
          const float ff = lk == lk ? f : 1.f;
          l += ff * lk;
          y.x += ff * v.x, y.y += ff * v.y, y.z += ff * v.z, y.w += ff * v.w;
        }
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store4<F32>(a.out, out_at(row) + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv), a.vec_out);
      } else {
        __stcg(reinterpret_cast<float4*>(part + row * HD + d), y);
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + C::kRows * HD + 2 * row), make_float2(mm, l));
      }
    }
    if (!whole) {
      // Parts are summed in CTA order, in two levels where there are many: the last to arrive of each run of kGroup
      // CTAs sums the run into its first slot, the last run to arrive sums the runs. Every load of a level is
      // independent of the others.
      const int c0 = (int)(item_at / per), c1 = (int)((item_at + it.stages - 1) / per), parts = c1 - c0 + 1;
      const bool two = parts > 2 * kGroup;  // a second level costs about as much as one more round of loads
      const int me = blockIdx.x, lead = two ? c0 + (me - c0) / kGroup * kGroup : c0;
      const int runs = two ? (parts + kGroup - 1) / kGroup : 1;
      const int run = two ? min(kGroup, c1 - lead + 1) : parts;  // parts of this CTA's run
      constexpr int kItems = (C::kRows * (HD / 4) + kConsumers - 1) / kConsumers;
      auto slot_of = [&](int k) { return a.part + (size_t)(2 * k + (k == c0)) * C::kRows * (HD + 2); };
      auto last_of = [&](int* count, int n) {  // this CTA's parts are written; true in the last of n to say so
        __threadfence();
        named_sync(1, kConsumers);
        if (tid == 0) {
          const int old = atomicAdd(count, 1);
          s_last = old == n - 1;
          if (old == n - 1) atomicExch(count, 0);  // as the next launch expects it
          __threadfence();
        }
        named_sync(1, kConsumers);
        return s_last != 0;
      };
      // the sum of n slots, from `from` on, `step` CTAs apart: maximum, sum and output of this thread's values
      float mm[kItems], ll[kItems];
      float4 y[kItems];
      auto gather = [&](int from, int step, int n) {
#pragma unroll
        for (int q = 0; q < kItems; q++) {
          const int i = tid + q * kConsumers, row = i / (HD / 4), d = (i % (HD / 4)) * 4;
          mm[q] = -kInf, ll[q] = 0.f, y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row >= row_n) continue;
          for (int k0 = 0; k0 < n; k0 += kGroup) {
            float2 ml[kGroup];
            float4 v[kGroup];
#pragma unroll
            for (int k = 0; k < kGroup; k++)
              if (k0 + k < n) {
                const float* p = slot_of(from + (k0 + k) * step);
                ml[k] = __ldcg(reinterpret_cast<const float2*>(p + C::kRows * HD + 2 * row));
                v[k] = __ldcg(reinterpret_cast<const float4*>(p + row * HD + d));
              } else {
                ml[k] = make_float2(-kInf, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
            float now = mm[q];
#pragma unroll
            for (int k = 0; k < kGroup; k++) now = fmaxf(now, ml[k].x);
            const float go = ll[q] != ll[q] ? 1.f : mm[q] == -kInf ? 0.f : exp2_fast(mm[q] - now);
            mm[q] = now;
            ll[q] *= go;
            y[q].x *= go, y[q].y *= go, y[q].z *= go, y[q].w *= go;
#pragma unroll
            for (int k = 0; k < kGroup; k++) {
              const float f = ml[k].y != ml[k].y ? 1.f : ml[k].x == -kInf ? 0.f : exp2_fast(ml[k].x - now);
              ll[q] = fmaf(ml[k].y, f, ll[q]);
              y[q].x = fmaf(v[k].x, f, y[q].x), y[q].y = fmaf(v[k].y, f, y[q].y);
              y[q].z = fmaf(v[k].z, f, y[q].z), y[q].w = fmaf(v[k].w, f, y[q].w);
            }
          }
        }
      };
      bool final = last_of(a.count + 2 * lead + (lead == c0), run);
      if (final && runs > 1) {
        gather(lead, 1, run);
        named_sync(1, kConsumers);  // everyone has read the slot that the sum goes to
        float* p = slot_of(lead);
#pragma unroll
        for (int q = 0; q < kItems; q++) {
          const int i = tid + q * kConsumers, row = i / (HD / 4), d = (i % (HD / 4)) * 4;
          if (row >= row_n) continue;
          __stcg(reinterpret_cast<float4*>(p + row * HD + d), y[q]);
          if (d == 0) __stcg(reinterpret_cast<float2*>(p + C::kRows * HD + 2 * row), make_float2(mm[q], ll[q]));
        }
        final = last_of(a.count + 2 * gridDim.x + c0, runs);
      }
      if (final) {
        gather(c0, runs > 1 ? kGroup : 1, runs > 1 ? runs : run);
#pragma unroll
        for (int q = 0; q < kItems; q++) {
          const int i = tid + q * kConsumers, row = i / (HD / 4), d = (i % (HD / 4)) * 4;
          if (row >= row_n) continue;
          const float inv = ll[q] == 0.f ? 0.f : 1.f / ll[q];
          store4<F32>(a.out, out_at(row) + d, make_float4(y[q].x * inv, y[q].y * inv, y[q].z * inv, y[q].w * inv), a.vec_out);
        }
      }
    }
    named_sync(1, kConsumers);  // the join buffer and the query fragments are free
    if (stage == it.stages) {
      stage = -kItemCost;
      if (w < w1) next_item();
    }
  }
}

template <int HD, int NG, int NT, bool F32>
int launch_one(coli_ctx* ctx, AttnArgs& a, long long most_stages) {
  using C = Cfg<HD, NG, NT, F32>;
  int grid = ctx->num_sms * C::kCtas;
  if (most_stages < grid) grid = (int)most_stages;
  if (grid > kKvCounters / 3) grid = kKvCounters / 3;
  static_assert((size_t)2 * C::kCtas * C::kRows * (HD + 2) <= kKvPartFloats, "an SM's CTAs leave more than there is room for");
  int rc = ensure_kv_part(ctx);
  if (rc != COLI_OK) return rc;
  a.part = ctx->d_kv_part;
  auto kern = kv4_attn_kernel<HD, NG, NT, F32>;
  static std::atomic<uint64_t> ready{0};  // devices (below 64) on which this instance has its attribute
  const uint64_t bit = ctx->device < 64 ? 1ull << ctx->device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_attention attribute");
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  ProfScope prof(ctx, COLI_KERNEL_ATTENTION);
  cudaError_t e = launch_k(kern, grid, kAttnThreads, C::kSmem, ctx->stream, true, false, a);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "kv4_attention launch");
  return COLI_OK;
}

// Query rows per tile: enough for the rows that a sequence has on average, since a tile's padding costs
// instructions and each further tile reads the cache again. Widths beyond the registers are cut into tiles.
template <int HD, int NG, bool F32>
int launch_rows(coli_ctx* ctx, AttnArgs& a) {
  const long long rows = (long long)((a.p.T + a.p.B - 1) / a.p.B) * a.group;
  const long long width = ((long long)a.p.table_stride << a.c.page_log2) / kStageTok + 1;
  auto most = [&](int nt) { return ((long long)a.p.T * a.group / (8 * nt) + a.p.B) * a.c.heads * width; };
  if (rows <= 8) return launch_one<HD, NG, 1, F32>(ctx, a, most(1));
  return launch_one<HD, NG, 2, F32>(ctx, a, most(2));
}

template <bool F32>
int launch_shape(coli_ctx* ctx, AttnArgs& a) {
  const int ng = a.c.ng;
  if (a.c.hd == 64) return ng == 1 ? launch_rows<64, 1, F32>(ctx, a) : launch_rows<64, 2, F32>(ctx, a);
  if (a.c.hd == 128)
    return ng == 1   ? launch_rows<128, 1, F32>(ctx, a)
           : ng == 2 ? launch_rows<128, 2, F32>(ctx, a)
                     : launch_rows<128, 4, F32>(ctx, a);
  return ng == 2 ? launch_rows<256, 2, F32>(ctx, a) : launch_rows<256, 4, F32>(ctx, a);
}

}  // namespace

}  // namespace coli
